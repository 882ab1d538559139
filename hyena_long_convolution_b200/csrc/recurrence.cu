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
// second half is the launch's number in 64 bits, which no earlier record has; 16
// bytes are written and read at once, so a record needs no flag or fence beside
// it.  The reader looks at the last 16 units together: from the nearest known
// carry it applies the units' (P, A) in order, the operations each unit itself
// performs, so the result does not depend on what was ready.  The gradient runs
// the same from the right.
//
// 10 bytes a channel-token forward, 18 for the gradient, 77 and 143 instructions
// a channel pair's token: HBM-bound where a device full of CTAs (three an SM forward, by
// their registers, two for the gradient, by its registers and its 106 KB of shared memory
// each) is a unit or two a chain, else bound by the carry's way from unit to unit.
// B x L x D, of the measured copy bandwidth (a range: two boards):
//   8 x 4096 x 4096   forward 223-230 us, 91-94%   gradient 446 us, 84%
//   2 x 8192 x 4096           142 us, 73%                   252 us, 75%
//   1 x 32768 x 4096          314-326 us, 64-66%            514 us, 73%
//   1 x 1024 x 4096            18 us, 36%
// The tile: 64 channels make rows of 128 bytes (narrower boxes read HBM slower);
// 64 tokens are 8 a warp, whose a and u stay in registers between the two sweeps.
// Units in clusters of four CTAs that pass their sums on through shared memory
// took 372 us for 1 x 32768 x 4096 and 309 us for 8 x 4096 x 4096 (a cluster
// waits for its slowest CTA); three passes over the data 1654 us.
#include <type_traits>

#include "recurrence_device.cuh"

namespace hyena {

namespace {

constexpr int kStages = 2;
constexpr int kTileBytes = RT * RCH * 2;  // one tensor's rows of a unit
constexpr int kParamBytes = RCH * 4;      // one fp32 value a channel
constexpr int kBatch = 4;                 // units whose records a look-back loads at a time

// A unit's rows of one tensor in shared memory as a lane sees them from its
// segment's first token: word i holds its channel pair of token i.
struct TileRows {
    uint32_t *p;
    __device__ __forceinline__ uint32_t operator()(int i) const { return p[i * (RCH / 2)]; }
};

__device__ __forceinline__ TileRows tile_rows(unsigned char *stage, int k, int warp, int lane)
{
    return TileRows{reinterpret_cast<uint32_t *>(stage + k * kTileBytes) + warp * RSEG * (RCH / 2) + lane};
}

// ---------------------------------------------------------------- records

struct Record {
    float2 v;
    unsigned long long tag;
};

__device__ __forceinline__ Record load_record(const uint4 *p)
{
    unsigned long long lo, hi;
    asm volatile("{\n\t.reg .b128 t;\n\tld.relaxed.gpu.global.b128 t, [%2];\n\tmov.b128 {%0, %1}, t;\n\t}"
                 : "=l"(lo), "=l"(hi)
                 : "l"(p)
                 : "memory");
    return Record{make_float2(__uint_as_float(static_cast<uint32_t>(lo)),
                              __uint_as_float(static_cast<uint32_t>(lo >> 32))),
                  hi};
}

__device__ __forceinline__ void store_record(uint4 *p, float2 v, unsigned long long tag)
{
    const unsigned long long lo =
        __float_as_uint(v.x) | static_cast<unsigned long long>(__float_as_uint(v.y)) << 32;
    asm volatile("{\n\t.reg .b128 t;\n\tmov.b128 t, {%1, %2};\n\tst.relaxed.gpu.global.b128 [%0], t;\n\t}" ::"l"(p),
                 "l"(lo), "l"(tag)
                 : "memory");
}

// What a unit publishes, a record a channel pair each: its P, its A, and the
// carry behind it.  Unit j of a chain in processing order is tile j chains +
// chain.
enum { kRecP, kRecA, kRecCarry };

struct Records {
    uint4 *base;  // [tiles][3][RCH / 2]
    int chains, chain, lane;
    unsigned long long epoch;

    __device__ __forceinline__ uint4 *at(int j, int kind) const
    {
        return base + ((static_cast<size_t>(j) * chains + chain) * 3 + kind) * (RCH / 2);
    }

    __device__ __forceinline__ void publish_unit(int j, float2 P, float2 A) const
    {
        store_record(at(j, kRecP) + lane, P, epoch);
        store_record(at(j, kRecA) + lane, A, epoch);
    }
    __device__ __forceinline__ void publish_carry(int j, float2 C) const
    {
        store_record(at(j, kRecCarry) + lane, C, epoch);
    }

    // Looking for the carry into unit j > 0, by all lanes of a warp.  glance():
    // the carry behind the unit before, and by one load more the first records of
    // the last 16 units, lanes 0-15 their carries, lanes 16-31 their sums.
    // look_back(): with what that brought, true if the carry can be formed: where
    // the nearest is not there yet, from the nearest that is, once every unit
    // behind it is there; each lane then loads its own channels' records.  The tag
    // of every record that is used is checked.
    struct Glance {
        Record nearest;
        unsigned long long first;  // its tag
    };
    struct Spot {  // what a unit's glances look at, worked out once
        const uint4 *nearest, *first;
        bool there;
    };
    __device__ __forceinline__ Spot spot(int j) const
    {
        const int back = lane & 15;
        return Spot{at(max(j - 1, 0), kRecCarry) + lane, at(max(j - 1 - back, 0), lane < 16 ? kRecCarry : kRecA),
                    back < j};
    }
    __device__ __forceinline__ Glance glance(const Spot &s) const
    {
        return Glance{load_record(s.nearest), load_record(s.first).tag};
    }
    __device__ __forceinline__ bool look_back(int j, const Spot &s, const Glance &g, float2 &C) const
    {
        C = g.nearest.v;
        if (__all_sync(kFullMask, g.nearest.tag == epoch)) return true;
        const unsigned int ready = __ballot_sync(kFullMask, s.there && g.first == epoch);
        const unsigned int units = ready >> 16;
        const int k = __ffs(ready & 0xffffu) - 1;  // nearest known carry
        if (k < 0 || ((units + 1u) & ((1u << k) - 1u)) != 0u) return false;
        // the carry and the kBatch farthest units behind it in one round trip to L2,
        // which a loop from the first batch on would make two
        const uint4 *from = at(j - 1 - k, kRecCarry) + lane;
        const Record r = load_record(from);
        Sums u;
        load_sums(j - k, j - 1, u);
        C = r.v;
        bool found = r.tag == epoch;
        apply(min(k, kBatch), u, C, found);
        for (int d = k - kBatch; d > 0; d -= kBatch) {
            load_sums(j - d, j - 1, u);
            apply(min(d, kBatch), u, C, found);
        }
        return __all_sync(kFullMask, found);
    }

    // Of kBatch units from `first` on (the last one again behind `last`), and their
    // first n applied to C.
    struct Sums {
        Record P[kBatch], A[kBatch];
    };
    __device__ __forceinline__ void load_sums(int first, int last, Sums &u) const
    {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            u.P[i] = load_record(at(min(first + i, last), kRecP) + lane);
            u.A[i] = load_record(at(min(first + i, last), kRecA) + lane);
        }
    }
    __device__ __forceinline__ void apply(int n, const Sums &u, float2 &C, bool &found) const
    {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (i < n) {
                found = found && u.P[i].tag == epoch && u.A[i].tag == epoch;
                C = carry<true>(u.P[i].v, C, u.A[i].v);
            }
        }
    }
};

// ---------------------------------------------------------------- work items

// The parameter k of a lane's channel pair; lanes without channels read what
// the shared memory holds, and write nothing.
__device__ __forceinline__ float2 param(const unsigned char *params, int k, int lane)
{
    return reinterpret_cast<const float2 *>(params + k * kParamBytes)[lane];
}

// Tokens behind the sequence's end, as the last unit's copy holds them (zeros):
// a gate of -inf makes them pass the state on as it is (a = 1), and x1 = -0
// their input -0, which adds nothing to any value, -0 neither.
__device__ __forceinline__ void pad_tail(const TileRows &x1, const TileRows &gate, int n)
{
    for (int i = max(n, 0); i < RSEG; ++i) {
        x1.p[i * (RCH / 2)] = 0x80008000u;
        gate.p[i * (RCH / 2)] = 0xff80ff80u;
    }
}

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
        *reinterpret_cast<unsigned long long *>(A.hdr + kRecEpoch) += 1u;
    }
}

// A tile: place j in processing order of a chain, the chain's batch row and
// first channel.  j < 0: no more tiles.
struct Tile {
    int j, chain, b, c;
};

__device__ __forceinline__ Tile tile_of(const RecArgs &A, unsigned int ticket)
{
    Tile t{-1, 0, 0, 0};
    if (ticket < A.tiles) {
        t.j = static_cast<int>(ticket / static_cast<unsigned int>(A.chains));
        t.chain = static_cast<int>(ticket - static_cast<unsigned int>(t.j) * A.chains);
        t.b = t.chain / A.nCB;
        t.c = (t.chain - t.b * A.nCB) * RCH;
    }
    return t;
}

// What forward and gradient share: two stages of N tensors' rows and the
// channels' parameters, their tiles and barriers.  Outputs go straight to global
// memory, a warp 128 bytes of a row at a time (as TMA stores from the stage,
// eight small ones a tensor, they cost the gradient 10%), so a stage takes new
// rows as soon as the warps are through with the tile.
template <int N, bool kBack>
struct Pipeline {
    static constexpr int kBytes = N * kTileBytes + 3 * kParamBytes;  // rows; log_rate, Dskip, start states
    Tile tile[kStages];
    uint64_t full[kStages];
    uint64_t sums, carried;  // of the current tile: the segments' sums, the carry into it
    uint64_t freed;          // the previous tile's stage
    unsigned int *error;

    // One thread.  A tile that is none only ends the wait for it.
    __device__ __forceinline__ void request(const RecMaps &m, const RecArgs &A, unsigned char *stages, int s, Tile t)
    {
        tile[s] = t;
        if (t.j < 0) {
            mbar_arrive(&full[s]);
            return;
        }
        const int unit = kBack ? A.units - 1 - t.j : t.j;
        unsigned char *stage = stages + s * kBytes, *params = stage + N * kTileBytes;
        const uint32_t bytes = 4u * min(RCH, A.D - t.c);  // a multiple of 32: D is one of 8
        mbar_arrive_expect_tx(&full[s], N * kTileBytes + bytes * (1 + (A.Dskip != nullptr) + kBack));
#pragma unroll
        for (int k = 0; k < N; ++k) tma_load_4d(stage + k * kTileBytes, &m.in[k], &full[s], t.c, 0, unit * RT, t.b);
        bulk_load(params, A.log_rate + t.c, bytes, &full[s]);
        if (A.Dskip != nullptr) bulk_load(params + kParamBytes, A.Dskip + t.c, bytes, &full[s]);
        if (kBack)
            bulk_load(params + 2 * kParamBytes,
                      A.unit_states + (static_cast<size_t>(t.b) * A.units + unit) * A.D + t.c, bytes, &full[s]);
    }
    __device__ __forceinline__ void start(const RecMaps &m, const RecArgs &A, unsigned char *stages)
    {
        for (int s = 0; s < kStages; ++s) mbar_init(&full[s], 1);
        mbar_init(&sums, RWARPS);
        mbar_init(&carried, 1);
        mbar_init(&freed, RWARPS);
        error = A.hdr + 2;
        fence_mbar_init();
        for (int s = 0; s < kStages; ++s) request(m, A, stages, s, tile_of(A, next_tile(A, s)));
    }
    // By a whole warp.  Longer than a look-back waits, so that one that gives up does
    // not put the CTA's own warps out of step; false if the wait ran out.  The warp
    // then has to leave: no barrier that it counts for completes again, so that none
    // is taken for a later phase, and the others' waits run out as well.
    __device__ __forceinline__ bool wait(uint64_t *bar, int turn)
    {
        if (__all_sync(kFullMask, mbar_try_wait(bar, turn & 1))) return true;
        unsigned long long t0 = global_timer_ns();
        for (int left = 4; left > 0;) {  // one span that passed while the CTA was suspended is not the end
            if (__all_sync(kFullMask, mbar_try_wait(bar, turn & 1))) return true;
            const unsigned long long now = global_timer_ns();
            if (__any_sync(kFullMask, now - t0 > kWaitLimitNs)) {
                t0 = now;
                --left;
            }
        }
        atomicOr(error, kErrLocalTimeout);
        return false;
    }
    // A computing warp's wait.  (A return value that its loops test took the forward
    // of 8 x 4096 x 4096 from 223 to 227 us.)
    __device__ __forceinline__ void wait_or_leave(uint64_t *bar, int turn)
    {
        if (!wait(bar, turn)) asm volatile("exit;");
    }
    // This warp's part of a barrier that counts warps.
    __device__ __forceinline__ void arrive(uint64_t *bar, int lane)
    {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    }
};

// A CTA: RWARPS warps that compute, and one that takes tickets, asks for rows
// and finds the carries, so that the computing warps' registers do not have to
// hold its work too.
constexpr int kThreads = (RWARPS + 1) * 32;

// The control warp.  What differs between forward and gradient is its Work:
//   sums()       from the segments' sums of tile t: P and A of its unit
//   initial(c)   the carry into the first unit;  known(t, C, E)  what else to
//                write once the carry C into the unit and E behind it are known
//   parts(t, s)  once tile t in stage s is done;  lost(t)  in a tile's place
// What a wait that runs out leaves behind is NaN, so that no result passes for
// one.  Behind a carry that was not found: all that it reaches.  Where a wait for
// the CTA's own warps or copies ran out: the CTA's tiles from then on; rows that
// one of its warps writes meanwhile are right (it left if its own wait had failed).
template <int N, bool kBack, class Work>
__device__ __forceinline__ void control_warp(Pipeline<N, kBack> &pipe, const RecMaps &maps, const RecArgs &A,
                                             unsigned char *stages, float2 *carry_in, int lane, Work work)
{
    const float nan = __int_as_float(0x7fffffff);
    Records rec{A.records, A.chains, 0, lane, 0u};
    if (A.units > 1) rec.epoch = *reinterpret_cast<const volatile unsigned long long *>(A.hdr + kRecEpoch) + 1u;
    Tile before{};
    unsigned int next = ~0u;  // the ticket of the tile after the stages'
    bool asked = true;
    int it = 0;
    for (;; ++it) {
        const int st = it % kStages;
        const Tile t = pipe.tile[st];
        asked = it == 0;
        if (t.j < 0) {
            if (it > 0) {
                if (!pipe.wait(&pipe.freed, it - 1)) break;
                work.parts(before, st ^ 1);
            }
            if (lane == 0) finish(A);
            return;
        }
        bool summed = false, found = t.j == 0;
        if (!asked && lane == 0) next = next_tile(A, it + 1);
        const auto ask = [&] {  // the tile before is done: its stage takes the next one's rows
            work.parts(before, st ^ 1);
            if (lane == 0) pipe.request(maps, A, stages, st ^ 1, tile_of(A, next));
            __syncwarp();
            asked = true;
        };
        float2 C = found ? work.initial(t) : bcast2(0.f), P, a;
        const bool last = t.j == A.units - 1;
        rec.chain = t.chain;
        const Records::Spot spot = rec.spot(t.j);
        unsigned long long t0 = 0;
        bool ok = true;
        for (;;) {
            // the glance's load is under way while the CTA's own barriers are looked at
            Records::Glance seen{};
            if (!found) seen = rec.glance(spot);
            if (!asked && __all_sync(kFullMask, mbar_test_wait(&pipe.freed, (it - 1) & 1))) ask();
            if (!summed) {
                if (found && !(ok = pipe.wait(&pipe.sums, it))) break;
                summed = found || __all_sync(kFullMask, mbar_test_wait(&pipe.sums, it & 1));
                if (summed) {
                    work.sums(st, P, a);
                    if (!found && !last) rec.publish_unit(t.j, P, a);
                }
            }
            if (!found) found = rec.look_back(t.j, spot, seen, C);
            if (found && summed) break;
            const unsigned long long now = global_timer_ns();
            if (t0 == 0) t0 = now;
            if (!found && __any_sync(kFullMask, now - t0 > kWaitLimitNs)) {
                if (lane == 0) atomicOr(pipe.error, kErrLookbackTimeout);
                C = bcast2(nan);
                found = true;
                if (summed) break;
            }
        }
        if (!ok) break;
        const float2 E = carry<true>(P, C, a);
        if (!last) rec.publish_carry(t.j, E);
        carry_in[lane] = C;
        // `freed` of the tile before is looked at before `carried`: it is complete, as a
        // warp frees that tile before it adds its sums of this one, and from `carried` on
        // the warps may complete this tile's too, whose parity is that of none before
        if (!asked && !pipe.wait(&pipe.freed, it - 1)) break;
        pipe.arrive(&pipe.carried, lane);
        work.known(t, C, E);
        if (!asked) ask();
        before = t;
    }
    // The CTA is given up: its tiles (both stages', one whose rows were not asked for,
    // and those that it draws from here on) are lost.  It works from another address of
    // the arguments, so that no value is held for it through the loop above (which
    // took the gradient of 1 x 32768 x 4096 from 514 to 534 us).
    const RecArgs *args = &A;
    asm volatile("" : "+l"(args));
    const Work cold = work.on(*args);
    Records gone{args->records, args->chains, 0, lane, rec.epoch};
    const int st = it % kStages, other = asked ? it + 1 : it - 1;
    mbar_wait_bounded(&pipe.full[st], it / kStages & 1);  // its copies are over
    if (other >= 0) mbar_wait_bounded(&pipe.full[st ^ 1], other / kStages & 1);
    __syncwarp();
#pragma unroll 1
    for (int k = asked ? 1 : 0, turn = it + 2;; ++k) {  // next; the stages'; from there on
        Tile t;
        if (k == 1 || k == 2) {
            t = pipe.tile[k - 1];
        } else {
            if (k > 2 && lane == 0) next = next_tile(*args, turn++);
            t = tile_of(*args, __shfl_sync(kFullMask, next, 0));
        }
        if (t.j < 0 && k > 2) break;
        if (t.j < 0) continue;
        gone.chain = t.chain;
        gone.publish_carry(t.j, bcast2(nan));
        cold.known(t, bcast2(nan), bcast2(nan));
        cold.lost(t);
    }
    if (lane == 0) finish(*args);
}

// NaN in the rows of a unit of a bf16 tensor, by one warp: a lane its channel
// pair.
__device__ __forceinline__ void lose_rows(uint16_t *p, long long ld, const RecArgs &A, const Tile &t, int unit,
                                          int lane)
{
    const int c = t.c + 2 * lane;
    if (c >= A.D) return;
    p += (static_cast<long long>(t.b) * A.L + unit * RT) * ld + c;
#pragma unroll 1
    for (int i = 0; i < min(A.L - unit * RT, RT); ++i, p += ld) *reinterpret_cast<uint32_t *>(p) = 0x7fff7fffu;
}

// ---------------------------------------------------------------- forward

// The segments' sums take the place of the first gates of each warp's own rows.
struct ForwardSums {
    float2 P[32], A[32], l[32];
};
static_assert(sizeof(ForwardSums) <= RSEG * RCH * 2, "a segment's sums fit in its rows of one tensor");

struct ForwardShared {
    float2 C[32];  // the carry into the tile
    Pipeline<4, false> pipe;
};

__device__ __forceinline__ ForwardSums &forward_sums(unsigned char *stage, int warp)
{
    return *reinterpret_cast<ForwardSums *>(stage + 3 * kTileBytes + warp * RSEG * RCH * 2);
}

template <bool kNorm, bool kReset>
__device__ __forceinline__ void forward_tile(ForwardShared &sh, const RecArgs &A, const Tile &t, int row,
                                             unsigned char *stage, int warp, int lane, int n, unsigned int mask,
                                             int it)
{
    const bool skip = A.Dskip != nullptr;
    const TileRows x1 = tile_rows(stage, 0, warp, lane), x2 = tile_rows(stage, 1, warp, lane);
    const TileRows x3 = tile_rows(stage, 2, warp, lane), gate = tile_rows(stage, 3, warp, lane);
    const unsigned char *params = stage + 4 * kTileBytes;
    if (n < RSEG) pad_tail(x1, gate, n);
    float2 a[RSEG], u[RSEG], l, P;
    segment_gates<kNorm, kReset>(a, u, l, P, gate, finite_rate(param(params, 0, lane)), mask);
#pragma unroll
    for (int i = 0; i < RSEG; ++i) {
        const float2 v = product(x1(i), x2(i));
        u[i] = kNorm ? __fmul2_rn(u[i], v) : v;
    }
    ForwardSums &own = forward_sums(stage, warp);
    __syncwarp();  // the warp has read its gates
    own.l[lane] = l;
    own.P[lane] = P;
    own.A[lane] = segment_end<kReset>(a, u, mask);
    fence_proxy_async_smem();  // before the stage's next rows
    sh.pipe.arrive(&sh.pipe.sums, lane);
    sh.pipe.wait_or_leave(&sh.pipe.carried, it);
    float2 C = sh.C[lane];
#pragma unroll
    for (int w = 0; w < RWARPS - 1; ++w) {
        if (w < warp) {
            const ForwardSums &f = forward_sums(stage, w);
            C = carry<kReset>(f.P[lane], C, f.A[lane]);
        }
    }
    const float2 dsk = skip ? param(params, 1, lane) : bcast2(0.f);
    const int m_out = t.c + 2 * lane < A.D ? n : 0;  // tokens that this lane writes
    uint16_t *y = A.y + (static_cast<long long>(t.b) * A.L + row) * A.ld_y + t.c + 2 * lane;
    const auto write = [&](auto whole) {  // the warp writes all of its rows: no test at each
#pragma unroll
        for (int i = 0; i < RSEG; ++i) {
            C = kReset && (mask >> i & 1u) ? u[i] : __ffma2_rn(a[i], C, u[i]);
            float2 o = __fmul2_rn(bf16x2_to_float2(x3(i)), C);
            if (skip) o = __ffma2_rn(dsk, product(x1(i), x2(i)), o);
            if (decltype(whole)::value || i < m_out) *reinterpret_cast<uint32_t *>(y) = float2_to_bf16x2(o);
            y += A.ld_y;
        }
    };
    if (__all_sync(kFullMask, m_out == RSEG))
        write(std::true_type());
    else
        write(std::false_type());
}

template <bool kReset>
struct ForwardWork {
    const RecArgs &A;
    unsigned char *stages;
    int lane;

    __device__ __forceinline__ size_t state(Tile t) const { return static_cast<size_t>(t.b) * A.D + t.c + 2 * lane; }
    __device__ __forceinline__ bool live(Tile t) const { return t.c + 2 * lane < A.D; }
    __device__ __forceinline__ float2 initial(Tile t) const
    {
        return A.state_in != nullptr && live(t) ? *reinterpret_cast<const float2 *>(A.state_in + state(t))
                                                : bcast2(0.f);
    }
    __device__ __forceinline__ void sums(int st, float2 &P, float2 &a) const
    {
        unsigned char *stage = stages + st * Pipeline<4, false>::kBytes;
        float2 l = forward_sums(stage, 0).l[lane];
        a = forward_sums(stage, 0).A[lane];
#pragma unroll
        for (int w = 1; w < RWARPS; ++w) {
            const ForwardSums &f = forward_sums(stage, w);
            l = __fadd2_rn(l, f.l[lane]);
            a = carry<kReset>(f.P[lane], a, f.A[lane]);
        }
        P = decay_over(l);
    }
    __device__ __forceinline__ void known(Tile t, float2 C, float2 E) const
    {
        if (!live(t)) return;
        if (A.C != nullptr)
            *reinterpret_cast<float2 *>(A.C + (static_cast<size_t>(t.b) * A.units + t.j) * A.D + t.c + 2 * lane) = C;
        if (t.j == A.units - 1 && A.state_out != nullptr)
            *reinterpret_cast<float2 *>(A.state_out + state(t)) = E;
    }
    __device__ __forceinline__ void parts(Tile, int) const {}
    __device__ __forceinline__ ForwardWork on(const RecArgs &a) const { return {a, stages, lane}; }
    __device__ __forceinline__ void lost(Tile t) const { lose_rows(A.y, A.ld_y, A, t, t.j, lane); }
};

template <bool kNorm, bool kReset>
__global__ void __launch_bounds__(kThreads, 3)
    recurrence_kernel(const __grid_constant__ RecMaps maps, const __grid_constant__ RecArgs A)
{
    extern __shared__ __align__(128) unsigned char stages[];
    __shared__ ForwardShared sh;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == RWARPS * 32) sh.pipe.start(maps, A, stages);
    __syncthreads();
    if (warp == RWARPS) {
        control_warp(sh.pipe, maps, A, stages, sh.C, lane, ForwardWork<kReset>{A, stages, lane});
        return;
    }
    for (int it = 0;; ++it) {
        const int st = it % kStages;
        sh.pipe.wait_or_leave(&sh.pipe.full[st], it / kStages);
        const Tile t = sh.pipe.tile[st];
        if (t.j < 0) break;
        unsigned char *stage = stages + st * sh.pipe.kBytes;
        const int n = min(A.L - t.j * RT - warp * RSEG, RSEG);  // tokens of the segment; it may have none
        const unsigned int mask =
            kReset ? segment_resets(A.reset, static_cast<long long>(t.b) * A.L + t.j * RT + warp * RSEG, n, lane) : 0u;
        forward_tile<kNorm, kReset>(sh, A, t, t.j * RT + warp * RSEG, stage, warp, lane, n, mask, it);
        sh.pipe.arrive(&sh.pipe.freed, lane);
    }
}

// ---------------------------------------------------------------- gradient

struct BackwardShared {
    float2 P[kStages][RWARPS][32], A[kStages][RWARPS][32], Q[kStages][RWARPS][32], l[kStages][RWARPS][32];
    float2 rate[kStages][RWARPS][32], skip[kStages][RWARPS][32];
    float2 E[32];  // the carry into the tile, from the right
    Pipeline<5, true> pipe;
};

template <bool kNorm, bool kReset>
__device__ __forceinline__ void backward_tile(BackwardShared &sh, const RecArgs &A, const Tile &t, int row,
                                              unsigned char *stage, int st, int warp, int lane, int n,
                                              unsigned int mask, int it)
{
    const bool skip = A.Dskip != nullptr;
    const TileRows x1 = tile_rows(stage, 0, warp, lane), x2 = tile_rows(stage, 1, warp, lane);
    const TileRows x3 = tile_rows(stage, 2, warp, lane), gate = tile_rows(stage, 3, warp, lane);
    const TileRows dy = tile_rows(stage, 4, warp, lane);
    const unsigned char *params = stage + 5 * kTileBytes;
    if (n < RSEG) pad_tail(x1, gate, n);
    const float2 rate = finite_rate(param(params, 0, lane));
    float2 a[RSEG], w[RSEG], prev[RSEG], l, P;
    segment_gates<kNorm, kReset>(a, w, l, P, gate, rate, mask);
#pragma unroll
    for (int i = 0; i < RSEG; ++i) {
        prev[i] = product(x1(i), x2(i));  // u, until the states are known
        if constexpr (kNorm) prev[i] = __fmul2_rn(w[i], prev[i]);
    }
    sh.l[st][warp][lane] = l;
    sh.P[st][warp][lane] = P;
    sh.A[st][warp][lane] = segment_end<kReset>(a, prev, mask);
    sh.Q[st][warp][lane] = segment_left<kReset>(a, x3, dy, mask);
    sh.pipe.arrive(&sh.pipe.sums, lane);
    // the state before each token, while the carry from the right is found
    sh.pipe.wait_or_leave(&sh.pipe.sums, it);
    float2 S = param(params, 2, lane);
#pragma unroll
    for (int k = 0; k < RWARPS - 1; ++k)
        if (k < warp) S = carry<kReset>(sh.P[st][k][lane], S, sh.A[st][k][lane]);
#pragma unroll
    for (int i = 0; i < RSEG; ++i) {
        const float2 s = kReset && (mask >> i & 1u) ? prev[i] : __ffma2_rn(a[i], S, prev[i]);
        prev[i] = S;
        S = s;
    }
    sh.pipe.wait_or_leave(&sh.pipe.carried, it);
    const float2 dsk = skip ? param(params, 1, lane) : bcast2(0.f);
    float2 e = sh.E[lane], d_rate = bcast2(0.f), d_skip = bcast2(0.f);
#pragma unroll
    for (int k = RWARPS - 1; k > 0; --k)
        if (k > warp) e = carry<kReset>(sh.P[st][k][lane], e, sh.Q[st][k][lane]);
    const int m_out = t.c + 2 * lane < A.D ? n : 0;  // tokens that this lane writes
    const long long at = static_cast<long long>(t.b) * A.L + row + RSEG - 1;
    uint16_t *o1 = A.dx1 + at * A.ld_dx + t.c + 2 * lane, *o2 = A.dx2 + at * A.ld_dx + t.c + 2 * lane;
    uint16_t *o3 = A.dx3 + at * A.ld_dx + t.c + 2 * lane, *og = A.dgate + at * A.ld_dg + t.c + 2 * lane;
    const auto write = [&](auto whole) {  // the warp writes all of its rows: no test at each
#pragma unroll
        for (int i = RSEG - 1; i >= 0; --i) {
            const bool cut = kReset && (mask >> i & 1u);
            const uint32_t w1 = x1(i), w2 = x2(i), wd = dy(i);
            const float2 d = bf16x2_to_float2(wd);
            const float2 v = product(w1, w2);
            const float2 q = fma_bf16x2(x3(i), wd, e);
            const bool put = decltype(whole)::value || i < m_out;
            if (put) *reinterpret_cast<uint32_t *>(o3) = float2_to_bf16x2(__fmul2_rn(d, S));
            float2 dv = kNorm ? __fmul2_rn(w[i], q) : q;
            if (skip) dv = __ffma2_rn(dsk, d, dv);
            if (put) {
                *reinterpret_cast<uint32_t *>(o1) = float2_to_bf16x2(__fmul2_rn(dv, bf16x2_to_float2(w2)));
                *reinterpret_cast<uint32_t *>(o2) = float2_to_bf16x2(__fmul2_rn(dv, bf16x2_to_float2(w1)));
            }
            o1 -= A.ld_dx;
            o2 -= A.ld_dx;
            o3 -= A.ld_dx;
            e = __fmul2_rn(a[i], q);
            float2 m = prev[i];
            S = m;
            if constexpr (kNorm) {
                // d w / d l = -a^2 / w; no gradient where w = 0 (log_rate = 0)
                const float2 r = make_float2(w[i].x > 0.f ? rcp_approx(w[i].x) : 0.f,
                                             w[i].y > 0.f ? rcp_approx(w[i].y) : 0.f);
                const float2 av = __fmul2_rn(a[i], v);
                m = __ffma2_rn(make_float2(-av.x, -av.y), r, m);
            }
            float2 dl = __fmul2_rn(e, m);
            if (cut) dl = e = bcast2(0.f);
            float2 eg;
            const float2 sig = gate_sigmoid(bf16x2_to_float2(gate(i)), eg);
            // not behind the end: dl there is finite only where the last state is
            if (decltype(whole)::value || i < n) d_rate = __ffma2_rn(dl, sig, d_rate);
            d_skip = __ffma2_rn(d, v, d_skip);
            // sig' = sig (1 - sig), with 1 - sig = exp(-gate) sig; 0 where the exponential overflows
            eg = make_float2(fminf(eg.x, 1e38f), fminf(eg.y, 1e38f));
            const float2 slope = __fmul2_rn(__fmul2_rn(eg, sig), sig);
            if (put) *reinterpret_cast<uint32_t *>(og) = float2_to_bf16x2(__fmul2_rn(__fmul2_rn(rate, dl), slope));
            og -= A.ld_dg;
        }
    };
    if (__all_sync(kFullMask, m_out == RSEG))
        write(std::true_type());
    else
        write(std::false_type());
    sh.rate[st][warp][lane] = d_rate;
    sh.skip[st][warp][lane] = d_skip;
}

template <bool kReset>
struct BackwardWork {
    const RecArgs &A;
    const BackwardShared &sh;
    int lane;

    __device__ __forceinline__ size_t state(Tile t) const { return static_cast<size_t>(t.b) * A.D + t.c + 2 * lane; }
    __device__ __forceinline__ bool live(Tile t) const { return t.c + 2 * lane < A.D; }
    __device__ __forceinline__ float2 initial(Tile t) const
    {
        return A.dstate_out != nullptr && live(t) ? *reinterpret_cast<const float2 *>(A.dstate_out + state(t))
                                                  : bcast2(0.f);
    }
    __device__ __forceinline__ void sums(int st, float2 &P, float2 &q) const
    {
        float2 l = sh.l[st][0][lane];
#pragma unroll
        for (int w = 1; w < RWARPS; ++w) l = __fadd2_rn(l, sh.l[st][w][lane]);
        q = sh.Q[st][RWARPS - 1][lane];
#pragma unroll
        for (int w = RWARPS - 2; w >= 0; --w) q = carry<kReset>(sh.P[st][w][lane], q, sh.Q[st][w][lane]);
        P = decay_over(l);
    }
    __device__ __forceinline__ void known(Tile t, float2, float2 E) const
    {
        if (live(t) && t.j == A.units - 1 && A.dstate_in != nullptr)
            *reinterpret_cast<float2 *>(A.dstate_in + state(t)) = E;
    }
    // The unit's parts of dlog_rate and dDskip replace its (P, A) record, with a
    // tag that no launch has: by then the unit's carry is published, and a reader
    // that finds no (P, A) looks again and finds the carry.
    __device__ __forceinline__ void parts(Tile t, int st) const
    {
        float2 d_rate = sh.rate[st][0][lane], d_skip = sh.skip[st][0][lane];
#pragma unroll
        for (int w = 1; w < RWARPS; ++w) {
            d_rate = __fadd2_rn(d_rate, sh.rate[st][w][lane]);
            d_skip = __fadd2_rn(d_skip, sh.skip[st][w][lane]);
        }
        uint4 *u = A.records + (static_cast<size_t>(t.j) * A.chains + t.chain) * (3 * RCH / 2) + lane;
        store_record(u + kRecP * (RCH / 2), d_rate, 0u);
        store_record(u + kRecA * (RCH / 2), d_skip, 0u);
    }
    __device__ __forceinline__ BackwardWork on(const RecArgs &a) const { return {a, sh, lane}; }
    __device__ __forceinline__ void lost(Tile t) const
    {
        const int unit = A.units - 1 - t.j;
        uint16_t *const rows[] = {A.dx1, A.dx2, A.dx3};
#pragma unroll 1
        for (int k = 0; k < 3; ++k) lose_rows(rows[k], A.ld_dx, A, t, unit, lane);
        lose_rows(A.dgate, A.ld_dg, A, t, unit, lane);
        const float2 nan = bcast2(__int_as_float(0x7fffffff));
        uint4 *u = A.records + (static_cast<size_t>(t.j) * A.chains + t.chain) * (3 * RCH / 2) + lane;
        store_record(u + kRecP * (RCH / 2), nan, 0u);
        store_record(u + kRecA * (RCH / 2), nan, 0u);
    }
};

template <bool kNorm, bool kReset>
__global__ void __launch_bounds__(kThreads, 2)
    recurrence_backward_kernel(const __grid_constant__ RecMaps maps, const __grid_constant__ RecArgs A)
{
    extern __shared__ __align__(128) unsigned char stages[];
    __shared__ BackwardShared sh;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == RWARPS * 32) sh.pipe.start(maps, A, stages);
    __syncthreads();
    if (warp == RWARPS) {
        control_warp(sh.pipe, maps, A, stages, sh.E, lane, BackwardWork<kReset>{A, sh, lane});
        return;
    }
    for (int it = 0;; ++it) {
        const int st = it % kStages;
        sh.pipe.wait_or_leave(&sh.pipe.full[st], it / kStages);
        const Tile t = sh.pipe.tile[st];
        if (t.j < 0) break;
        unsigned char *stage = stages + st * sh.pipe.kBytes;
        const int unit = A.units - 1 - t.j;
        const int n = min(A.L - unit * RT - warp * RSEG, RSEG);  // tokens of the segment; it may have none
        const unsigned int mask =
            kReset ? segment_resets(A.reset, static_cast<long long>(t.b) * A.L + unit * RT + warp * RSEG, n, lane) : 0u;
        backward_tile<kNorm, kReset>(sh, A, t, unit * RT + warp * RSEG, stage, st, warp, lane, n, mask, it);
        if (n < RSEG) fence_proxy_async_smem();  // what pad_tail wrote, before the stage's next rows
        sh.pipe.arrive(&sh.pipe.freed, lane);
    }
}

// dlog_rate and dDskip: the units' parts summed in double, in a fixed order: a
// CTA takes one of the two for a chain's channels over all batch rows and
// units, each of its 32 warps every 32nd part, a lane a channel pair; then the
// warps by butterfly.  Latency-bound, so that a thread's loads go out together
// (2 x 8192 x 4096: 6.6 us, one load at a time 11).
__global__ void __launch_bounds__(1024) unit_sum_kernel(const RecArgs A)
{
    __shared__ double sum[32][2 * 32 + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int kind = blockIdx.x & 1, cb = blockIdx.x >> 1;
    float *out = kind == kRecP ? A.dlog_rate : A.dDskip;
    if (out == nullptr) return;
    const unsigned int parts = static_cast<unsigned int>(A.B) * A.units;  // below 2^31, as the tiles are
    double x = 0., y = 0.;
    // tile j chains + b nCB + cb is (j B + b) nCB + cb
    const uint4 *first = A.records + (static_cast<size_t>(cb) * 3 + kind) * (RCH / 2) + lane;
#pragma unroll 8
    for (unsigned int k = warp; k < parts; k += 32) {
        const float2 q = *reinterpret_cast<const float2 *>(first + static_cast<size_t>(k) * A.nCB * (3 * RCH / 2));
        x += q.x;
        y += q.y;
    }
    sum[warp][2 * lane] = x;
    sum[warp][2 * lane + 1] = y;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // two channels a warp, a lane a warp's sum
        double v = sum[lane][2 * warp + i];
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kFullMask, v, d);
        const int c = cb * RCH + 2 * warp + i;
        if (lane == 0 && c < A.D) out[c] = static_cast<float>(v);
    }
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
    const float2 v =
        product(*reinterpret_cast<const uint32_t *>(A.x1 + o), *reinterpret_cast<const uint32_t *>(A.x2 + o));
    const float2 f3 = bf16x2_to_float2(*reinterpret_cast<const uint32_t *>(A.x3 + o));
    const float2 g = bf16x2_to_float2(*reinterpret_cast<const uint32_t *>(A.gate + b * A.ld_g + c));
    float2 *st = reinterpret_cast<float2 *>(A.state_out + static_cast<size_t>(b) * A.D + c);
    const float2 S = *st;
    float2 a, w, e;
    decay<kNorm>(__fmul2_rn(finite_rate(ldg_f2(A.log_rate + c)), gate_sigmoid(g, e)), a, w);
    const float2 s = __ffma2_rn(a, S, kNorm ? __fmul2_rn(w, v) : v);
    *st = s;
    float2 y = __fmul2_rn(f3, s);
    if (A.Dskip != nullptr) y = __ffma2_rn(ldg_f2(A.Dskip + c), v, y);
    *reinterpret_cast<uint32_t *>(A.y + b * A.ld_y + c) = float2_to_bf16x2(y);
}

// One persistent CTA per free place on the device, at most one per tile.
template <auto kernel>
int launch_units(int tensors, const RecMaps &maps, const RecArgs &a, cudaStream_t st)
{
    thread_local int configured_device = -1, places = 0;  // per kernel and thread
    const int smem = kStages * (tensors * kTileBytes + 3 * kParamBytes);
    int dev = 0;
    HYENA_TRY(cudaGetDevice(&dev), "gated recurrence: current device");
    if (configured_device != dev) {
        int sms = 0, per_sm = 0;
        HYENA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem),
                  "gated recurrence: set max dynamic shared memory");
        HYENA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev), "multiprocessor count");
        HYENA_TRY(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kThreads, smem),
                  "gated recurrence: occupancy");
        places = sms * (per_sm > 0 ? per_sm : 1);
        configured_device = dev;
    }
    const unsigned int grid = a.tiles < static_cast<unsigned int>(places) ? a.tiles : places;
    kernel<<<grid, kThreads, smem, st>>>(maps, a);
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
