// recurrence.cu -- the gated linear recurrence and its gradient on sm_100a:
// the recurrence of the modal scan with one mode per channel whose pole depends
// on the token.
//
//   l_t = log_rate sigmoid(gate_t);  a_t = exp(l_t), 0 at a reset
//   s_t = a_t s_{t-1} + w_t v_t,  v = x1 x2,  w_t = sqrt(1 - a_t^2) or 1
//   y_t = x3_t s_t + Dskip v_t
// and, from dy and the gradient of the last state,
//   q_t = x3_t dy_t + e_{t+1},  e_t = a_t q_t        (right to left)
//   dx3 = dy s;  dv = w q + Dskip dy;  dx1 = dv x2;  dx2 = dv x1
//   dl  = a q (s_{t-1} - a v / w), the second term with w = sqrt(1 - a^2) only,
//         0 at a reset;  dgate = dl log_rate sig (1 - sig)
//   dlog_rate = sum dl sig;  dDskip = sum dy v;  dstate_in = e_0
//
// Time is cut into units of RT tokens of RCH channels, one CTA's work item: a
// warp takes a segment of RSEG tokens, a lane a channel pair.  A unit maps the
// state at its start to the one at its end by C <- P C + A (P its decay, A its
// end state from zero), evaluated in fp32 in the same way wherever a sequence
// is cut, so chunks of whole units reproduce the single pass bit for bit.
//
// One pass over the data: a CTA reads a unit once (TMA into shared memory, the
// next unit's rows while this one is computed), forms (P, A), takes the carry
// from the units before it and writes its outputs from the same copy.  Units
// are handed out in time-major order by an atomic ticket, so the unit a CTA
// waits for is always running or done.  A unit publishes 16-byte records whose
// third word is the launch's epoch; 16 bytes are written and read at once, so a
// record needs no flag or fence beside it.  The reader looks at the last
// kLookBack units together: from the nearest known carry it applies the units'
// (P, A) in order, the operations each unit itself performs, so the result does
// not depend on what was ready.  The gradient runs the same from the right.
#include "recurrence_device.cuh"

namespace hyena {

namespace {

constexpr int kStages = 2;
constexpr int kTileBytes = RT * RCH * 2;  // one tensor's rows of a unit
constexpr int kLookBack = 4;

// A unit's rows of one tensor in shared memory as a lane sees them from its
// segment's first token: word i holds its channel pair of token i.
struct TileRows {
    const uint32_t *p;
    __device__ __forceinline__ uint32_t operator()(int i) const { return p[i * (RCH / 2)]; }
};

__device__ __forceinline__ TileRows tile_rows(const unsigned char *stage, int k, int warp, int lane)
{
    return TileRows{reinterpret_cast<const uint32_t *>(stage + k * kTileBytes) + warp * RSEG * (RCH / 2) + lane};
}

// ---------------------------------------------------------------- records

__device__ __forceinline__ uint4 load_record(const uint4 *p)
{
    unsigned long long lo, hi;
    asm volatile("{\n\t.reg .b128 t;\n\tld.relaxed.gpu.global.b128 t, [%2];\n\tmov.b128 {%0, %1}, t;\n\t}"
                 : "=l"(lo), "=l"(hi)
                 : "l"(p)
                 : "memory");
    return make_uint4(static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32), static_cast<uint32_t>(hi),
                      static_cast<uint32_t>(hi >> 32));
}

__device__ __forceinline__ void store_record(uint4 *p, float a, float b, uint32_t tag)
{
    const unsigned long long lo =
        __float_as_uint(a) | static_cast<unsigned long long>(__float_as_uint(b)) << 32;
    const unsigned long long hi = tag;
    asm volatile("{\n\t.reg .b128 t;\n\tmov.b128 t, {%1, %2};\n\tst.relaxed.gpu.global.b128 [%0], t;\n\t}" ::"l"(p),
                 "l"(lo), "l"(hi)
                 : "memory");
}

// What a unit publishes: per channel (P, A), per channel pair the carry behind
// it.  Unit j of a chain in processing order is tile j chains + chain.
struct Records {
    uint4 *unit;   // [tiles][RCH]
    uint4 *carry;  // [tiles][RCH / 2]
    int chains, chain, lane;
    uint32_t epoch;

    __device__ __forceinline__ size_t tile(int j) const { return static_cast<size_t>(j) * chains + chain; }
    __device__ __forceinline__ void publish_unit(int j, float2 P, float2 A) const
    {
        uint4 *u = unit + tile(j) * RCH + 2 * lane;
        store_record(u, P.x, A.x, epoch);
        store_record(u + 1, P.y, A.y, epoch);
    }
    __device__ __forceinline__ void publish_carry(int j, float2 C) const
    {
        store_record(carry + tile(j) * (RCH / 2) + lane, C.x, C.y, epoch);
    }

    // The carry into unit j > 0 (all lanes of a warp).  Gives up after the
    // bounded wait, with an error bit, and returns zero.
    __device__ __forceinline__ float2 carry_into(int j, unsigned int *error) const
    {
        const unsigned long long t0 = global_timer_ns();
        for (;;) {
            uint4 c[kLookBack], u0[kLookBack - 1], u1[kLookBack - 1];
#pragma unroll
            for (int d = 0; d < kLookBack; ++d) {
                const int i = max(j - 1 - d, 0);
                c[d] = load_record(carry + tile(i) * (RCH / 2) + lane);
                if (d < kLookBack - 1) {
                    u0[d] = load_record(unit + tile(i) * RCH + 2 * lane);
                    u1[d] = load_record(unit + tile(i) * RCH + 2 * lane + 1);
                }
            }
            float2 C = bcast2(0.f);
            // nearest known carry, then forward over the units between
            int k = kLookBack;
#pragma unroll
            for (int d = kLookBack - 1; d >= 0; --d)
                if (j - 1 - d >= 0 && c[d].z == epoch) k = d;
            bool found = k < kLookBack;
#pragma unroll
            for (int d = kLookBack - 1; d >= 0; --d) {
                if (d == k) C = make_float2(__uint_as_float(c[d].x), __uint_as_float(c[d].y));
                if (d < kLookBack - 1 && d < k) {
                    found = found && u0[d].z == epoch && u1[d].z == epoch;
                    C = hyena::carry(make_float2(__uint_as_float(u0[d].x), __uint_as_float(u1[d].x)), C,
                                     make_float2(__uint_as_float(u0[d].y), __uint_as_float(u1[d].y)));
                }
            }
            if (__all_sync(kFullMask, found)) return C;
            if (global_timer_ns() - t0 > kWaitLimitNs) {
                if (lane == 0) atomicOr(error, kErrLookbackTimeout);
                return bcast2(0.f);
            }
        }
    }
};

// ---------------------------------------------------------------- work items

// The next tile of this CTA (called by one thread).  Sequences of one unit have
// nothing to wait for and need no ticket.
__device__ __forceinline__ unsigned int next_tile(const RecArgs &A, int turn)
{
    if (A.units == 1) return blockIdx.x + static_cast<unsigned int>(turn) * gridDim.x;
    return atomicAdd(A.hdr, 1u);
}

// The last CTA leaves the tickets and the epoch ready for the next launch.
__device__ __forceinline__ void finish(const RecArgs &A)
{
    if (A.units == 1) return;
    if (atomicAdd(A.hdr + 1, 1u) + 1u == gridDim.x) {
        A.hdr[0] = 0u;
        A.hdr[1] = 0u;
        A.hdr[3] += 1u;
    }
}

// Where a warp's lane works in a tile.
struct Place {
    int b, j, unit, c;    // batch row, place in processing order, unit, first channel of the pair
    int n, nseg;          // tokens of the segment; segments of the unit that hold tokens
    long long row;        // b L + t of the segment's first token
    bool live;            // the channel pair exists
};

template <bool kBack>
__device__ __forceinline__ Place place_of(const RecArgs &A, unsigned int tile, int warp, int lane)
{
    Place p;
    p.j = static_cast<int>(tile / static_cast<unsigned int>(A.chains));
    const int chain = static_cast<int>(tile - static_cast<unsigned int>(p.j) * A.chains);
    p.unit = kBack ? A.units - 1 - p.j : p.j;
    p.b = chain / A.nCB;
    p.c = (chain - p.b * A.nCB) * RCH + 2 * lane;
    p.live = p.c < A.D;
    if (!p.live) p.c = 0;  // reads a channel that exists, writes nothing
    const int t0 = p.unit * RT;
    const int rows = min(RT, A.L - t0);
    p.nseg = (rows + RSEG - 1) / RSEG;
    p.n = min(max(rows - warp * RSEG, 0), RSEG);
    p.row = static_cast<long long>(p.b) * A.L + t0 + warp * RSEG;
    return p;
}

// Requests a tile's rows of N tensors; one thread.
template <int N, bool kBack>
__device__ __forceinline__ void request(const RecMaps &m, const RecArgs &A, unsigned int tile, unsigned char *stage,
                                        uint64_t *bar)
{
    const int j = static_cast<int>(tile / static_cast<unsigned int>(A.chains));
    const int chain = static_cast<int>(tile - static_cast<unsigned int>(j) * A.chains);
    const int b = chain / A.nCB;
    const int c = (chain - b * A.nCB) * RCH;
    const int t = (kBack ? A.units - 1 - j : j) * RT;
    mbar_arrive_expect_tx(bar, N * kTileBytes);
#pragma unroll
    for (int k = 0; k < N; ++k) tma_load_4d(stage + k * kTileBytes, &m.m[k], bar, c, 0, t, b);
}

__device__ __forceinline__ uint32_t output_pair(float2 x3, float2 s, bool skip, float2 dsk, float2 v)
{
    const float2 o = __fmul2_rn(x3, s);
    return float2_to_bf16x2(skip ? __ffma2_rn(dsk, v, o) : o);
}

// ---------------------------------------------------------------- forward

struct ForwardShared {
    float2 P[RWARPS][32], l[RWARPS][32], A[RWARPS][32];
    float2 C[32];
    uint64_t full[kStages];
    unsigned int tile[kStages];
};

template <bool kNorm, bool kReset>
__global__ void __launch_bounds__(RWARPS * 32, 3)
    recurrence_kernel(const __grid_constant__ RecMaps maps, const RecArgs A)
{
    extern __shared__ __align__(128) unsigned char stages[];
    __shared__ ForwardShared sh;
    constexpr int N = 4;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Records rec{A.rec_unit, A.rec_carry, A.chains, 0, lane, 0u};
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) mbar_init(&sh.full[s], 1);
        fence_mbar_init();
        for (int s = 0; s < kStages; ++s) {
            sh.tile[s] = next_tile(A, s);
            if (sh.tile[s] < A.tiles) request<N, false>(maps, A, sh.tile[s], stages + s * N * kTileBytes, &sh.full[s]);
        }
    }
    if (A.units > 1) rec.epoch = ld_volatile_u32(A.hdr + 3) + 1u;
    __syncthreads();
    for (int it = 0;; ++it) {
        const int st = it % kStages;
        const unsigned int tile = sh.tile[st];
        if (tile >= A.tiles) break;
        const Place p = place_of<false>(A, tile, warp, lane);
        rec.chain = static_cast<int>(tile % static_cast<unsigned int>(A.chains));
        const unsigned char *stage = stages + st * N * kTileBytes;
        const TileRows x1 = tile_rows(stage, 0, warp, lane), x2 = tile_rows(stage, 1, warp, lane);
        const TileRows x3 = tile_rows(stage, 2, warp, lane), gate = tile_rows(stage, 3, warp, lane);
        const float2 rate = ldg_f2(A.log_rate + p.c);
        const float2 dsk = A.Dskip != nullptr ? ldg_f2(A.Dskip + p.c) : bcast2(0.f);
        const unsigned int mask = kReset ? segment_resets(A.reset, p.row, p.n, lane) : 0u;
        const size_t state = static_cast<size_t>(p.b) * A.D + p.c;
        if (!mbar_wait_bounded(&sh.full[st], (it / kStages) & 1) && threadIdx.x == 0)
            atomicOr(A.hdr + 2, kErrTmaTimeout);

        RecSegment s;
        segment_gates<kNorm, kReset>(s, gate, p.n, rate, mask);
        sh.l[warp][lane] = s.l;
        sh.P[warp][lane] = decay_over(s.l);
        sh.A[warp][lane] = segment_end<kNorm, kReset>(s, x1, x2, p.n, mask);
        __syncthreads();
        unsigned int next = 0;
        if (threadIdx.x == 32) next = next_tile(A, it + kStages);
        if (warp == 0) {
            float2 l = sh.l[0][lane], a = sh.A[0][lane];
#pragma unroll
            for (int w = 1; w < RWARPS; ++w) {
                if (w < p.nseg) {
                    l = __fadd2_rn(l, sh.l[w][lane]);
                    a = carry(sh.P[w][lane], a, sh.A[w][lane]);
                }
            }
            const float2 P = decay_over(l);
            const bool last = p.j == A.units - 1;
            float2 C = bcast2(0.f);
            if (p.j > 0) {
                if (!last) rec.publish_unit(p.j, P, a);
                C = rec.carry_into(p.j, A.hdr + 2);
            } else if (A.state_in != nullptr) {
                C = *reinterpret_cast<const float2 *>(A.state_in + state);
            }
            sh.C[lane] = C;
            const float2 E = carry(P, C, a);
            if (!last) rec.publish_carry(p.j, E);
            if (p.live) {
                if (A.C != nullptr)
                    *reinterpret_cast<float2 *>(A.C + (static_cast<size_t>(p.b) * A.units + p.unit) * A.D + p.c) = C;
                if (last && A.state_out != nullptr) *reinterpret_cast<float2 *>(A.state_out + state) = E;
            }
        }
        __syncthreads();
        float2 C = sh.C[lane];
#pragma unroll
        for (int w = 0; w < RWARPS - 1; ++w)
            if (w < warp) C = carry(sh.P[w][lane], C, sh.A[w][lane]);
        uint16_t *y = A.y + p.row * A.ld_y + p.c;
#pragma unroll
        for (int i = 0; i < RSEG; ++i) {
            if (i < p.n) {
                const float2 v = __fmul2_rn(bf16x2_to_float2(x1(i)), bf16x2_to_float2(x2(i)));
                const float2 u = kNorm ? __fmul2_rn(s.w[i], v) : v;
                C = kReset && (mask >> i & 1u) ? u : __ffma2_rn(s.a[i], C, u);
                const uint32_t o = output_pair(bf16x2_to_float2(x3(i)), C, A.Dskip != nullptr, dsk, v);
                if (p.live) *reinterpret_cast<uint32_t *>(y + i * A.ld_y) = o;
            }
        }
        __syncthreads();  // the stage and the segments' sums may be overwritten
        if (threadIdx.x == 32) {
            sh.tile[st] = next;
            if (next < A.tiles) {
                fence_proxy_async_smem();
                request<N, false>(maps, A, next, stages + st * N * kTileBytes, &sh.full[st]);
            }
        }
    }
    if (threadIdx.x == 0) finish(A);
}

// ---------------------------------------------------------------- gradient

struct BackwardShared {
    float2 P[RWARPS][32], l[RWARPS][32], A[RWARPS][32], Q[RWARPS][32];
    float2 rate[RWARPS][32], skip[RWARPS][32];
    float2 E[32];
    uint64_t full[kStages];
    unsigned int tile[kStages];
};

// The units' parts of dlog_rate and dDskip replace their (P, A) records, with
// a tag that no launch has: by then the unit's carry is published, and a reader
// that finds no (P, A) looks again and finds the carry.
template <bool kNorm, bool kReset>
__global__ void __launch_bounds__(RWARPS * 32, 2)
    recurrence_backward_kernel(const __grid_constant__ RecMaps maps, const RecArgs A)
{
    extern __shared__ __align__(128) unsigned char stages[];
    __shared__ BackwardShared sh;
    constexpr int N = 5;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Records rec{A.rec_unit, A.rec_carry, A.chains, 0, lane, 0u};
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) mbar_init(&sh.full[s], 1);
        fence_mbar_init();
        for (int s = 0; s < kStages; ++s) {
            sh.tile[s] = next_tile(A, s);
            if (sh.tile[s] < A.tiles) request<N, true>(maps, A, sh.tile[s], stages + s * N * kTileBytes, &sh.full[s]);
        }
    }
    if (A.units > 1) rec.epoch = ld_volatile_u32(A.hdr + 3) + 1u;
    __syncthreads();
    for (int it = 0;; ++it) {
        const int st = it % kStages;
        const unsigned int tile = sh.tile[st];
        if (tile >= A.tiles) break;
        const Place p = place_of<true>(A, tile, warp, lane);
        rec.chain = static_cast<int>(tile % static_cast<unsigned int>(A.chains));
        const unsigned char *stage = stages + st * N * kTileBytes;
        const TileRows x1 = tile_rows(stage, 0, warp, lane), x2 = tile_rows(stage, 1, warp, lane);
        const TileRows x3 = tile_rows(stage, 2, warp, lane), gate = tile_rows(stage, 3, warp, lane);
        const TileRows dy = tile_rows(stage, 4, warp, lane);
        const float2 rate = ldg_f2(A.log_rate + p.c);
        const float2 dsk = A.Dskip != nullptr ? ldg_f2(A.Dskip + p.c) : bcast2(0.f);
        const unsigned int mask = kReset ? segment_resets(A.reset, p.row, p.n, lane) : 0u;
        const size_t state = static_cast<size_t>(p.b) * A.D + p.c;
        float2 S = ldg_f2(A.unit_states + (static_cast<size_t>(p.b) * A.units + p.unit) * A.D + p.c);
        if (!mbar_wait_bounded(&sh.full[st], (it / kStages) & 1) && threadIdx.x == 0)
            atomicOr(A.hdr + 2, kErrTmaTimeout);

        RecSegment s;
        segment_gates<kNorm, kReset>(s, gate, p.n, rate, mask);
        sh.l[warp][lane] = s.l;
        sh.P[warp][lane] = decay_over(s.l);
        sh.A[warp][lane] = segment_end<kNorm, kReset>(s, x1, x2, p.n, mask);
        sh.Q[warp][lane] = segment_left<kReset>(s, x3, dy, p.n, mask);
        __syncthreads();
        unsigned int next = 0;
        if (threadIdx.x == 32) next = next_tile(A, it + kStages);
        if (warp == 0) {
            float2 l = sh.l[0][lane], q = sh.Q[p.nseg - 1][lane];
#pragma unroll
            for (int w = 1; w < RWARPS; ++w)
                if (w < p.nseg) l = __fadd2_rn(l, sh.l[w][lane]);
#pragma unroll
            for (int w = RWARPS - 2; w >= 0; --w)
                if (w < p.nseg - 1) q = carry(sh.P[w][lane], q, sh.Q[w][lane]);
            const float2 P = decay_over(l);
            const bool last = p.j == A.units - 1;
            float2 E = bcast2(0.f);
            if (p.j > 0) {
                if (!last) rec.publish_unit(p.j, P, q);
                E = rec.carry_into(p.j, A.hdr + 2);
            } else if (A.dstate_out != nullptr) {
                E = *reinterpret_cast<const float2 *>(A.dstate_out + state);
            }
            sh.E[lane] = E;
            const float2 out = carry(P, E, q);
            if (!last) rec.publish_carry(p.j, out);
            if (last && p.live && A.dstate_in != nullptr) *reinterpret_cast<float2 *>(A.dstate_in + state) = out;
        }
        // the states before the segment's tokens, meanwhile
#pragma unroll
        for (int w = 0; w < RWARPS - 1; ++w)
            if (w < warp) S = carry(sh.P[w][lane], S, sh.A[w][lane]);
        float2 prev[RSEG];
#pragma unroll
        for (int i = 0; i < RSEG; ++i) {
            if (i < p.n) {
                float2 u = __fmul2_rn(bf16x2_to_float2(x1(i)), bf16x2_to_float2(x2(i)));
                if constexpr (kNorm) u = __fmul2_rn(s.w[i], u);
                prev[i] = S;
                S = kReset && (mask >> i & 1u) ? u : __ffma2_rn(s.a[i], S, u);
            }
        }
        __syncthreads();
        float2 e = sh.E[lane];
#pragma unroll
        for (int w = RWARPS - 1; w > 0; --w)
            if (w > warp && w < p.nseg) e = carry(sh.P[w][lane], e, sh.Q[w][lane]);
        float2 d_rate = bcast2(0.f), d_skip = bcast2(0.f);
        uint16_t *dx1 = A.dx1 + p.row * A.ld_dx + p.c, *dx2 = A.dx2 + p.row * A.ld_dx + p.c;
        uint16_t *dx3 = A.dx3 + p.row * A.ld_dx + p.c, *dgate = A.dgate + p.row * A.ld_dg + p.c;
#pragma unroll
        for (int i = RSEG - 1; i >= 0; --i) {
            if (i < p.n) {
                const bool cut = kReset && (mask >> i & 1u);
                const float2 f1 = bf16x2_to_float2(x1(i)), f2 = bf16x2_to_float2(x2(i));
                const float2 f3 = bf16x2_to_float2(x3(i)), d = bf16x2_to_float2(dy(i));
                const float2 v = __fmul2_rn(f1, f2);
                const float2 q = __fadd2_rn(__fmul2_rn(f3, d), e);
                const float2 d3 = __fmul2_rn(d, S);
                float2 dv = kNorm ? __fmul2_rn(s.w[i], q) : q;
                if (A.Dskip != nullptr) dv = __ffma2_rn(dsk, d, dv);
                const float2 t = __fmul2_rn(s.a[i], q);
                float2 m = prev[i];
                if constexpr (kNorm) {
                    // d w / d l = -a^2 / w; no gradient where w = 0 (log_rate = 0)
                    const float2 r = make_float2(s.w[i].x > 0.f ? rcp_approx(s.w[i].x) : 0.f,
                                                 s.w[i].y > 0.f ? rcp_approx(s.w[i].y) : 0.f);
                    const float2 av = __fmul2_rn(s.a[i], v);
                    m = __ffma2_rn(make_float2(-av.x, -av.y), r, m);
                }
                float2 dl = __fmul2_rn(t, m);
                e = t;
                S = prev[i];
                if (cut) dl = e = bcast2(0.f);
                float2 eg;
                const float2 sig = gate_sigmoid(bf16x2_to_float2(gate(i)), eg);
                const float2 ds = __fmul2_rn(dl, sig);
                d_rate = __ffma2_rn(dl, sig, d_rate);
                d_skip = __ffma2_rn(d, v, d_skip);
                // sig' = sig (1 - sig), with 1 - sig = exp(-gate) sig
                const float2 dg = __fmul2_rn(__fmul2_rn(rate, ds), __fmul2_rn(eg, sig));
                if (p.live) {
                    *reinterpret_cast<uint32_t *>(dx1 + i * A.ld_dx) = float2_to_bf16x2(__fmul2_rn(dv, f2));
                    *reinterpret_cast<uint32_t *>(dx2 + i * A.ld_dx) = float2_to_bf16x2(__fmul2_rn(dv, f1));
                    *reinterpret_cast<uint32_t *>(dx3 + i * A.ld_dx) = float2_to_bf16x2(d3);
                    *reinterpret_cast<uint32_t *>(dgate + i * A.ld_dg) = float2_to_bf16x2(dg);
                }
            }
        }
        sh.rate[warp][lane] = d_rate;
        sh.skip[warp][lane] = d_skip;
        __syncthreads();  // the stage and the segments' sums may be overwritten
        if (threadIdx.x == 32) {
            sh.tile[st] = next;
            if (next < A.tiles) {
                fence_proxy_async_smem();
                request<N, true>(maps, A, next, stages + st * N * kTileBytes, &sh.full[st]);
            }
        }
        if (warp == 0) {  // the next writes of these sums follow a barrier that this warp is in
#pragma unroll
            for (int w = 1; w < RWARPS; ++w) {
                d_rate = __fadd2_rn(d_rate, sh.rate[w][lane]);
                d_skip = __fadd2_rn(d_skip, sh.skip[w][lane]);
            }
            uint4 *u = A.rec_unit + static_cast<size_t>(tile) * RCH + 2 * lane;
            store_record(u, d_rate.x, d_skip.x, 0u);
            store_record(u + 1, d_rate.y, d_skip.y, 0u);
        }
    }
    if (threadIdx.x == 0) finish(A);
}

// dlog_rate and dDskip: the units' parts summed in double, in a fixed order: 32
// channels a CTA, 32 warps of which each takes every 32nd part.
__global__ void __launch_bounds__(1024) unit_sum_kernel(const RecArgs A)
{
    __shared__ double sum[2][32][33];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int half = blockIdx.x & 1, cb = blockIdx.x >> 1;
    const long long parts = static_cast<long long>(A.B) * A.units;
    double r = 0., d = 0.;
    for (long long k = warp; k < parts; k += 32) {
        const long long j = k / A.B, b = k - j * A.B;
        const uint4 q = A.rec_unit[(static_cast<size_t>(j) * A.chains + b * A.nCB + cb) * RCH + half * 32 + lane];
        r += __uint_as_float(q.x);
        d += __uint_as_float(q.y);
    }
    sum[0][warp][lane] = r;
    sum[1][warp][lane] = d;
    __syncthreads();
    const int c = cb * RCH + half * 32 + lane;
    if (warp > 1 || c >= A.D) return;
    float *out = warp == 0 ? A.dlog_rate : A.dDskip;
    if (out == nullptr) return;
    double v = 0.;
    for (int w = 0; w < 32; ++w) v += sum[warp][w][lane];
    out[c] = static_cast<float>(v);
}

// One token per batch row: the scan's arithmetic on a unit of one token.
constexpr int kRecDecodeThreads = 64;

template <bool kNorm>
__global__ void __launch_bounds__(kRecDecodeThreads) recurrence_decode_kernel(const RecArgs A)
{
    const long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
    const int pairs = A.D / 2;
    if (i >= static_cast<long long>(A.B) * pairs) return;
    const int b = static_cast<int>(i / pairs);
    const int c = 2 * static_cast<int>(i - static_cast<long long>(b) * pairs);
    const long long o = b * A.ld_x + c;
    const float2 v = __fmul2_rn(bf16x2_to_float2(*reinterpret_cast<const uint32_t *>(A.x1 + o)),
                                bf16x2_to_float2(*reinterpret_cast<const uint32_t *>(A.x2 + o)));
    const float2 f3 = bf16x2_to_float2(*reinterpret_cast<const uint32_t *>(A.x3 + o));
    const float2 g = bf16x2_to_float2(*reinterpret_cast<const uint32_t *>(A.gate + b * A.ld_g + c));
    float2 *st = reinterpret_cast<float2 *>(A.state_out + static_cast<size_t>(b) * A.D + c);
    const float2 S = *st;
    const float2 dsk = A.Dskip != nullptr ? ldg_f2(A.Dskip + c) : bcast2(0.f);
    float2 a, w, e;
    decay<kNorm>(__fmul2_rn(ldg_f2(A.log_rate + c), gate_sigmoid(g, e)), a, w);
    const float2 s = __ffma2_rn(a, S, kNorm ? __fmul2_rn(w, v) : v);
    *st = s;
    *reinterpret_cast<uint32_t *>(A.y + b * A.ld_y + c) = output_pair(f3, s, A.Dskip != nullptr, dsk, v);
}

// One persistent CTA per free place on the device, at most one per tile.
template <auto kernel>
int launch_units(int tensors, const RecMaps &maps, const RecArgs &a, cudaStream_t st)
{
    thread_local int configured_device = -1, places = 0;  // per kernel and thread
    const int smem = kStages * tensors * kTileBytes;
    int dev = 0;
    HYENA_TRY(cudaGetDevice(&dev), "gated recurrence: current device");
    if (configured_device != dev) {
        int sms = 0, per_sm = 0;
        HYENA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem),
                  "gated recurrence: set max dynamic shared memory");
        HYENA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev), "multiprocessor count");
        HYENA_TRY(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, RWARPS * 32, smem),
                  "gated recurrence: occupancy");
        places = sms * (per_sm > 0 ? per_sm : 1);
        configured_device = dev;
    }
    const unsigned int grid = a.tiles < static_cast<unsigned int>(places) ? a.tiles : places;
    kernel<<<grid, RWARPS * 32, smem, st>>>(maps, a);
    HYENA_TRY(cudaGetLastError(), "gated recurrence launch");
    return 1;
}

}  // namespace

int launch_recurrence(const RecMaps &maps, const RecArgs &a, bool normalize, bool back, cudaStream_t st)
{
    const bool reset = a.reset != nullptr;
    if (!back) {
        if (normalize)
            return reset ? launch_units<recurrence_kernel<true, true>>(4, maps, a, st)
                         : launch_units<recurrence_kernel<true, false>>(4, maps, a, st);
        return reset ? launch_units<recurrence_kernel<false, true>>(4, maps, a, st)
                     : launch_units<recurrence_kernel<false, false>>(4, maps, a, st);
    }
    int n;
    if (normalize)
        n = reset ? launch_units<recurrence_backward_kernel<true, true>>(5, maps, a, st)
                  : launch_units<recurrence_backward_kernel<true, false>>(5, maps, a, st);
    else
        n = reset ? launch_units<recurrence_backward_kernel<false, true>>(5, maps, a, st)
                  : launch_units<recurrence_backward_kernel<false, false>>(5, maps, a, st);
    if (n < 0) return n;
    unit_sum_kernel<<<2 * a.nCB, 1024, 0, st>>>(a);
    HYENA_TRY(cudaGetLastError(), "gated recurrence gradient sums launch");
    return n + 1;
}

int launch_recurrence_decode(const RecArgs &a, bool normalize, cudaStream_t st)
{
    const long long n = static_cast<long long>(a.B) * (a.D / 2);
    const unsigned int grid = static_cast<unsigned int>((n + kRecDecodeThreads - 1) / kRecDecodeThreads);
    if (normalize)
        recurrence_decode_kernel<true><<<grid, kRecDecodeThreads, 0, st>>>(a);
    else
        recurrence_decode_kernel<false><<<grid, kRecDecodeThreads, 0, st>>>(a);
    HYENA_TRY(cudaGetLastError(), "gated recurrence decode launch");
    return 1;
}

}  // namespace hyena
