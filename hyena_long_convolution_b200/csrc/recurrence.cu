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
// Time is cut into units of RT tokens.  A unit maps the state at its start to
// the one at its end by C <- P C + A (P its decay, A its end state from zero),
// evaluated in fp32 in the same way wherever a sequence is cut, so chunks of
// whole units reproduce the single pass bit for bit.
#include "recurrence_device.cuh"

namespace hyena {

namespace {

// One tensor's rows as a lane sees them: word i holds its channel pair of token i.
struct GlobalRows {
    const uint16_t *p;
    long long ld;
    __device__ __forceinline__ uint32_t operator()(int i) const
    {
        return __ldg(reinterpret_cast<const uint32_t *>(p + i * ld));
    }
};

// Where a thread works: batch row, unit, segment, channel pair.
struct Place {
    int b, unit, c, warp, lane;
    int n;                // tokens of the segment
    int nseg;             // segments of the unit that hold tokens
    long long row;        // b L + t of the segment's first token
    bool live;            // the channel pair exists
};

__device__ __forceinline__ Place place_of(const RecArgs &A)
{
    Place p;
    const int tile = blockIdx.x;
    const int chain = tile % A.chains;
    p.unit = tile / A.chains;
    p.b = chain / A.nCB;
    p.warp = threadIdx.x >> 5;
    p.lane = threadIdx.x & 31;
    p.c = (chain % A.nCB) * RCH + 2 * p.lane;
    p.live = p.c < A.D;
    if (!p.live) p.c = 0;  // reads a channel that exists, writes nothing
    const int t0 = p.unit * RT;
    const int rows = min(RT, A.L - t0);
    p.nseg = (rows + RSEG - 1) / RSEG;
    p.n = min(max(rows - p.warp * RSEG, 0), RSEG);
    p.row = static_cast<long long>(p.b) * A.L + t0 + p.warp * RSEG;
    return p;
}

__device__ __forceinline__ size_t unit_index(const RecArgs &A, const Place &p)
{
    return (static_cast<size_t>(p.b) * A.units + p.unit) * A.D + p.c;
}

__device__ __forceinline__ GlobalRows rows_of(const uint16_t *x, long long ld, const Place &p)
{
    return GlobalRows{x + p.row * ld + p.c, ld};
}

// Pass 1, forward: every unit's (P, A); gradient: its (P, Q).
template <bool kNorm, bool kReset, bool kBack>
__global__ void __launch_bounds__(RWARPS * 32) unit_aggregate_kernel(const RecArgs A)
{
    __shared__ float2 sP[RWARPS][32], sL[RWARPS][32], sA[RWARPS][32];
    const Place p = place_of(A);
    const float2 rate = ldg_f2(A.log_rate + p.c);
    const unsigned int mask = kReset ? segment_resets(A.reset, p.row, p.n, p.lane) : 0u;
    RecSegment s;
    segment_gates<kNorm, kReset>(s, rows_of(A.gate, A.ld_g, p), p.n, rate, mask);
    sL[p.warp][p.lane] = s.l;
    sP[p.warp][p.lane] = decay_over(s.l);
    if constexpr (kBack)
        sA[p.warp][p.lane] =
            segment_left<kReset>(s, rows_of(A.x3, A.ld_x, p), rows_of(A.dy, A.ld_dy, p), p.n, mask);
    else
        sA[p.warp][p.lane] =
            segment_end<kNorm, kReset>(s, rows_of(A.x1, A.ld_x, p), rows_of(A.x2, A.ld_x, p), p.n, mask);
    __syncthreads();
    if (p.warp != 0 || !p.live) return;
    float2 l = sL[0][p.lane];
    for (int w = 1; w < p.nseg; ++w) l = __fadd2_rn(l, sL[w][p.lane]);
    float2 a;
    if constexpr (kBack) {
        a = sA[p.nseg - 1][p.lane];
        for (int w = p.nseg - 2; w >= 0; --w) a = carry(sP[w][p.lane], a, sA[w][p.lane]);
    } else {
        a = sA[0][p.lane];
        for (int w = 1; w < p.nseg; ++w) a = carry(sP[w][p.lane], a, sA[w][p.lane]);
    }
    *reinterpret_cast<float2 *>(A.P + unit_index(A, p)) = decay_over(l);
    *reinterpret_cast<float2 *>(A.A + unit_index(A, p)) = a;
}

// Pass 2: the carries, unit after unit (the gradient's from the right).
template <bool kBack>
__global__ void __launch_bounds__(128) unit_carry_kernel(const RecArgs A)
{
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= A.B * A.D) return;
    const int b = i / A.D, c = i % A.D;
    const float *in = kBack ? A.dstate_out : A.state_in;
    float *out = kBack ? A.dstate_in : A.state_out;
    float C = in != nullptr ? in[i] : 0.f;
    const size_t first = static_cast<size_t>(b) * A.units * A.D + c;
    for (int j = 0; j < A.units; ++j) {
        const size_t k = first + static_cast<size_t>(kBack ? A.units - 1 - j : j) * A.D;
        A.C[k] = C;
        C = carry1(A.P[k], C, A.A[k]);
    }
    if (out != nullptr) out[i] = C;
}

// Pass 3, forward: outputs from the unit's carry.
template <bool kNorm, bool kReset>
__global__ void __launch_bounds__(RWARPS * 32) unit_output_kernel(const RecArgs A)
{
    __shared__ float2 sP[RWARPS][32], sA[RWARPS][32];
    const Place p = place_of(A);
    const float2 rate = ldg_f2(A.log_rate + p.c);
    const unsigned int mask = kReset ? segment_resets(A.reset, p.row, p.n, p.lane) : 0u;
    const GlobalRows x1 = rows_of(A.x1, A.ld_x, p), x2 = rows_of(A.x2, A.ld_x, p), x3 = rows_of(A.x3, A.ld_x, p);
    RecSegment s;
    segment_gates<kNorm, kReset>(s, rows_of(A.gate, A.ld_g, p), p.n, rate, mask);
    sP[p.warp][p.lane] = decay_over(s.l);
    sA[p.warp][p.lane] = segment_end<kNorm, kReset>(s, x1, x2, p.n, mask);
    __syncthreads();
    if (p.n == 0 || !p.live) return;
    float2 C = ldg_f2(A.C + unit_index(A, p));
    for (int w = 0; w < p.warp; ++w) C = carry(sP[w][p.lane], C, sA[w][p.lane]);
    const float2 dsk = A.Dskip != nullptr ? ldg_f2(A.Dskip + p.c) : bcast2(0.f);
    uint16_t *y = A.y + p.row * A.ld_y + p.c;
#pragma unroll
    for (int i = 0; i < RSEG; ++i) {
        if (i < p.n) {
            const float2 v = __fmul2_rn(bf16x2_to_float2(x1(i)), bf16x2_to_float2(x2(i)));
            const float2 u = kNorm ? __fmul2_rn(s.w[i], v) : v;
            C = kReset && (mask >> i & 1u) ? u : __ffma2_rn(s.a[i], C, u);
            const float2 o = __ffma2_rn(dsk, v, __fmul2_rn(bf16x2_to_float2(x3(i)), C));
            *reinterpret_cast<uint32_t *>(y + i * A.ld_y) = float2_to_bf16x2(o);
        }
    }
}

// Pass 3, gradient: the inputs' gradients from the unit's start state and the
// carry from its right, and the unit's parts of dlog_rate and dDskip.
template <bool kNorm, bool kReset>
__global__ void __launch_bounds__(RWARPS * 32) unit_gradient_kernel(const RecArgs A)
{
    __shared__ float2 sP[RWARPS][32], sA[RWARPS][32], sQ[RWARPS][32];
    const Place p = place_of(A);
    const float2 rate = ldg_f2(A.log_rate + p.c);
    const unsigned int mask = kReset ? segment_resets(A.reset, p.row, p.n, p.lane) : 0u;
    const GlobalRows x1 = rows_of(A.x1, A.ld_x, p), x2 = rows_of(A.x2, A.ld_x, p), x3 = rows_of(A.x3, A.ld_x, p);
    const GlobalRows gate = rows_of(A.gate, A.ld_g, p), dy = rows_of(A.dy, A.ld_dy, p);
    RecSegment s;
    segment_gates<kNorm, kReset>(s, gate, p.n, rate, mask);
    sP[p.warp][p.lane] = decay_over(s.l);
    sA[p.warp][p.lane] = segment_end<kNorm, kReset>(s, x1, x2, p.n, mask);
    sQ[p.warp][p.lane] = segment_left<kReset>(s, x3, dy, p.n, mask);
    __syncthreads();
    float2 S = ldg_f2(A.unit_states + unit_index(A, p));
    for (int w = 0; w < p.warp; ++w) S = carry(sP[w][p.lane], S, sA[w][p.lane]);
    float2 e = ldg_f2(A.C + unit_index(A, p));
    for (int w = p.nseg - 1; w > p.warp; --w) e = carry(sP[w][p.lane], e, sQ[w][p.lane]);
    __syncthreads();
    const float2 dsk = A.Dskip != nullptr ? ldg_f2(A.Dskip + p.c) : bcast2(0.f);
    float2 prev[RSEG];  // the state before each token
#pragma unroll
    for (int i = 0; i < RSEG; ++i) {
        if (i < p.n) {
            const bool cut = kReset && (mask >> i & 1u);
            float2 u = __fmul2_rn(bf16x2_to_float2(x1(i)), bf16x2_to_float2(x2(i)));
            if constexpr (kNorm) u = __fmul2_rn(s.w[i], u);
            prev[i] = S;
            S = cut ? u : __ffma2_rn(s.a[i], S, u);
        }
    }
    float2 d_rate = bcast2(0.f), d_skip = bcast2(0.f);
#pragma unroll
    for (int i = RSEG - 1; i >= 0; --i) {
        if (i < p.n) {
            const bool cut = kReset && (mask >> i & 1u);
            const float2 f1 = bf16x2_to_float2(x1(i)), f2 = bf16x2_to_float2(x2(i));
            const float2 f3 = bf16x2_to_float2(x3(i)), d = bf16x2_to_float2(dy(i));
            const float2 v = __fmul2_rn(f1, f2);
            const float2 q = __fadd2_rn(__fmul2_rn(f3, d), e);
            const float2 dx3 = __fmul2_rn(d, S);
            const float2 dv = __ffma2_rn(dsk, d, kNorm ? __fmul2_rn(s.w[i], q) : q);
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
                const long long o = (p.row + i) * A.ld_dx + p.c;
                *reinterpret_cast<uint32_t *>(A.dx1 + o) = float2_to_bf16x2(__fmul2_rn(dv, f2));
                *reinterpret_cast<uint32_t *>(A.dx2 + o) = float2_to_bf16x2(__fmul2_rn(dv, f1));
                *reinterpret_cast<uint32_t *>(A.dx3 + o) = float2_to_bf16x2(dx3);
                *reinterpret_cast<uint32_t *>(A.dgate + (p.row + i) * A.ld_dg + p.c) = float2_to_bf16x2(dg);
            }
        }
    }
    sA[p.warp][p.lane] = d_rate;
    sQ[p.warp][p.lane] = d_skip;
    __syncthreads();
    if (p.warp != 0 || !p.live) return;
    for (int w = 1; w < RWARPS; ++w) {
        d_rate = __fadd2_rn(d_rate, sA[w][p.lane]);
        d_skip = __fadd2_rn(d_skip, sQ[w][p.lane]);
    }
    *reinterpret_cast<float2 *>(A.P + unit_index(A, p)) = d_rate;
    *reinterpret_cast<float2 *>(A.A + unit_index(A, p)) = d_skip;
}

// dlog_rate and dDskip: the units' parts summed in double, in order.
__global__ void __launch_bounds__(128) unit_sum_kernel(const RecArgs A)
{
    const int c = blockIdx.x * blockDim.x + threadIdx.x;
    if (c >= A.D) return;
    double r = 0., d = 0.;
    for (long long j = 0; j < static_cast<long long>(A.B) * A.units; ++j) {
        r += A.P[j * A.D + c];
        d += A.A[j * A.D + c];
    }
    A.dlog_rate[c] = static_cast<float>(r);
    if (A.dDskip != nullptr) A.dDskip[c] = static_cast<float>(d);
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
    *reinterpret_cast<uint32_t *>(A.y + b * A.ld_y + c) = float2_to_bf16x2(__ffma2_rn(dsk, v, __fmul2_rn(f3, s)));
}

template <bool kNorm, bool kReset>
void forward(const RecArgs &a, unsigned int tiles, unsigned int carries, cudaStream_t st)
{
    unit_aggregate_kernel<kNorm, kReset, false><<<tiles, RWARPS * 32, 0, st>>>(a);
    unit_carry_kernel<false><<<carries, 128, 0, st>>>(a);
    unit_output_kernel<kNorm, kReset><<<tiles, RWARPS * 32, 0, st>>>(a);
}

template <bool kNorm, bool kReset>
void backward(const RecArgs &a, unsigned int tiles, unsigned int carries, cudaStream_t st)
{
    unit_aggregate_kernel<kNorm, kReset, true><<<tiles, RWARPS * 32, 0, st>>>(a);
    unit_carry_kernel<true><<<carries, 128, 0, st>>>(a);
    unit_gradient_kernel<kNorm, kReset><<<tiles, RWARPS * 32, 0, st>>>(a);
    unit_sum_kernel<<<(a.D + 127) / 128, 128, 0, st>>>(a);
}

}  // namespace

int launch_recurrence(const RecArgs &a, bool normalize, bool back, cudaStream_t st)
{
    const unsigned int tiles = static_cast<unsigned int>(a.chains) * static_cast<unsigned int>(a.units);
    const unsigned int carries = static_cast<unsigned int>((static_cast<long long>(a.B) * a.D + 127) / 128);
    const int which = (back ? 4 : 0) + (normalize ? 2 : 0) + (a.reset != nullptr ? 1 : 0);
    switch (which) {
        case 0: forward<false, false>(a, tiles, carries, st); break;
        case 1: forward<false, true>(a, tiles, carries, st); break;
        case 2: forward<true, false>(a, tiles, carries, st); break;
        case 3: forward<true, true>(a, tiles, carries, st); break;
        case 4: backward<false, false>(a, tiles, carries, st); break;
        case 5: backward<false, true>(a, tiles, carries, st); break;
        case 6: backward<true, false>(a, tiles, carries, st); break;
        default: backward<true, true>(a, tiles, carries, st); break;
    }
    HYENA_TRY(cudaGetLastError(), "gated recurrence launch");
    return back ? 4 : 3;
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
