// layer_internal.h -- host-side declarations of the gated recurrence and the RMS
// norm, shared by their entry points and launchers (not part of the public
// interface).
#pragma once

#include "hyena_internal.h"

namespace hyena {

// ---------------------------------------------------------------- gated recurrence
// Units of RT tokens (HYENA_RECURRENCE_UNIT) of chains of RCH channels of one
// batch row; arrays per unit and channel are [B][units][D].
constexpr int RT = HYENA_RECURRENCE_UNIT;
constexpr int RCH = 64;
constexpr int RWARPS = 8;          // computing warps of a CTA, one time segment each
constexpr int RSEG = RT / RWARPS;  // tokens per segment

struct RecArgs {
    const uint16_t *x1, *x2, *x3, *gate, *dy;
    long long ld_x, ld_g, ld_dy;
    const float *log_rate, *Dskip;
    const uint8_t *reset;  // [B][L] or null
    uint16_t *y;
    long long ld_y;
    const float *state_in;  // [B][D] or null
    float *state_out;       // [B][D] or null (decode: the state, in place)
    const float *unit_states;  // gradient: state before each unit
    const float *dstate_out;
    float *dstate_in;
    uint16_t *dx1, *dx2, *dx3, *dgate;
    long long ld_dx, ld_dg;
    float *dlog_rate, *dDskip;
    int B, L, D;
    int nCB, chains, units;  // chains per batch row, B nCB, ceil(L / RT)
    unsigned int tiles;      // chains units
    float *C;                // forward: unit_states or null
    // workspace: header ([0] next ticket, [1] finished CTAs, [2] error bits,
    // [4..5] launches so far, the next one's epoch - 1), then 16-byte records, all
    // with their tag in the second half
    unsigned int *hdr;
    uint4 *records;          // [tiles][3][RCH / 2]: P, A (later the gradient's parts), carry
};
constexpr size_t kRecHeaderBytes = 256;
constexpr int kRecEpoch = 4;  // header word
constexpr size_t kRecTileBytes = (RCH + RCH / 2) * 16;

// Tensor maps [B][L][1][D] over x1, x2, x3, gate and (gradient) dy, boxes of RT
// tokens x RCH channels.
struct RecMaps {
    CUtensorMap in[5];
};

// Forward (or, with `back`, the gradient); the number of launches or -1.
int launch_recurrence(const RecMaps &maps, const RecArgs &a, bool normalize, bool back, cudaStream_t st);
int launch_recurrence_decode(const RecArgs &a, bool normalize, cudaStream_t st);

// ---------------------------------------------------------------- RMS norm
struct NormArgs {
    const uint16_t *x;  // forward
    long long ld_x;     // of x, and of dx
    const void *residual;
    void *residual_out;
    long long ld_r;     // of the residual, residual_out, dres_out
    int res_kind;       // 1 bf16, 2 fp32: type of the residual (gradient: of h)
    const void *weight;
    bool weight_bf16;
    float eps;
    uint16_t *y;        // bf16 output, or
    uint8_t *q;         // e4m3 output with
    float *scales;      // one scale per row (group 0) or per 128 channels
    int group;
    long long ld_y;     // of y or q, and of dy
    float *rstd;
    long long rows;
    int D;
    // gradient
    const uint16_t *dy;
    const void *h;
    long long ld_h;
    const float *rstd_in;
    const void *dres_out;
    uint16_t *dx;
    float *dres;        // fp32 only
    long long ld_dr;
    float *dweight;
    float *partial;     // workspace [norm_parts(rows, D)][D]
    int stages;         // of the kernel's ring, and whether dres_out goes through it
    bool stage_dres;
};

int launch_rms_norm(const NormArgs &a, cudaStream_t st);
int launch_rms_norm_backward(const NormArgs &a, cudaStream_t st);
int norm_parts(long long rows, int D);

}  // namespace hyena
