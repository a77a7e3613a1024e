// ssd_ops_internal.h -- interface between the host code of the short causal
// convolution and the selective scan (ssd_ops.cpp) and their kernels.  Host
// declarations only; not part of the ABI.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

namespace ssd {

// Elements between batch entries and between tokens.
struct Strides {
    int64_t batch, row;
};

// ---------------------------------------------------------------------------
// Short causal convolution (kc_conv.hip)
// ---------------------------------------------------------------------------

struct ConvArgs {
    int64_t batch;
    int seqlen, channels, width;
    bool silu;
    bool in_bf16, y_bf16, dx_bf16;  // x and states; y and dy; dx
    Strides xs, dys;
    const void *x;
    const float *weight, *bias;
    const void *init;        // initial state, or the step's state
    const int32_t *lengths;  // null: all seqlen
    void *y, *final_state;
    // backward
    const void *dy;
    const float *dfinal;
    void *dx;
    float *dweight, *dbias, *dinit;
    float *partials;  // (ConvBwdPlan::parts, width + 1, channels)
};

// The strips of tokens the backward pass cuts each sequence into, and how many
// rows of partial sums its blocks leave.
struct ConvBwdPlan {
    int strip;      // tokens of one wave, a multiple of 16
    int nstrips;    // strips of one sequence
    int64_t parts;  // batch * ceil(nstrips / 4)
};
ConvBwdPlan conv_bwd_plan(int64_t batch, int64_t seqlen, int64_t channels);

hipError_t launch_conv_fwd(const ConvArgs &a, hipStream_t stream);
hipError_t launch_conv_bwd(const ConvArgs &a, const ConvBwdPlan &plan, hipStream_t stream);
hipError_t launch_conv_step(const ConvArgs &a, hipStream_t stream);

// ---------------------------------------------------------------------------
// Selective scan (ks_scan.hip, ks_scan_bwd.hip)
// ---------------------------------------------------------------------------

// Each channel's states are spread over 2, 4, 8 or 16 lanes, 4 states a lane;
// a block of 256 threads holds 1024 / (padded states) channels.
inline int padded_states(int64_t dstate) { return dstate <= 8 ? 8 : dstate <= 16 ? 16 : dstate <= 32 ? 32 : 64; }

constexpr int kScanTile = 8;    // tokens between the states that the backward pass keeps
constexpr int kScanSegment = 16;  // segments start at multiples of this
constexpr int kScanRun = 256;     // most tokens that a sum in fp32 takes; those sums are added in 64 bits

struct ScanPlan {
    int np;           // padded states
    int gblocks;      // blocks of one group
    int nblk;         // blocks of one batch entry: ngroups * gblocks
    int nseg;         // segments of the time axis
    int seglen;       // tokens of one, a multiple of kScanSegment
    int runs;         // backward: sums over tokens that a segment leaves, one per kScanRun tokens
    int64_t tiles;    // tiles of kScanTile tokens in seqlen, rounded up to whole kScanSegments
};
ScanPlan scan_plan(int64_t batch, int64_t seqlen, int64_t channels, int64_t dstate, int64_t ngroups, bool backward);

struct ScanArgs {
    int64_t batch;
    int seqlen, channels, dstate, ngroups;
    bool in_bf16, y_bf16, softplus;
    Strides xs, dts, Bs, Cs, zs, dys;
    const void *x, *dt, *B, *C, *z;
    const float *A, *D, *dt_bias;
    const float *init;  // initial state, or the step's state
    const int32_t *lengths;
    void *y;
    float *final_state;
    // Segments (nseg > 1): first each segment's own end state, then in place
    // the state it starts from, (batch, nseg, channels, np); the sums of its
    // step sizes, (batch, nseg, channels).
    float *seg_state, *seg_steps;
    // backward
    const void *dy;
    const float *dfinal;
    float *dx, *ddt, *dA, *dB, *dC, *dD, *dz, *ddt_bias, *dinit;
    float *seg_adj;     // as seg_state, for the gradient at each segment's end
    float *tile_state;  // state before each tile, (batch, tiles, channels, np)
    float *tile_steps;  // sum of the segment's steps before each tile (nseg > 1)
    // partial dB, dC per block of a group, (nblk, batch, seqlen, dstate); reserved but not used where one block a
    // group writes dB and dC themselves
    float *dbp, *dcp;
    float *dap;         // partial dA, (batch, nseg, runs, channels, np)
    float *ddp, *dbiasp;  // partial dD and ddt_bias, (batch, nseg, runs, channels)
};

// The backward pass's last sums: eight threads an output.  A launch has fewer
// than 2^24 blocks of 256 threads (32 bits of threads); its blocks take groups
// of outputs in turn.
constexpr int kSumSlices = 8, kSumOutputs = 256 / kSumSlices;
struct ScanSums {
    int64_t rates;   // outputs of dA
    int64_t rows;    // of dB, of dC; 0 where one block a group wrote them in place
    int64_t groups;  // of kSumOutputs outputs
    unsigned blocks;
};
inline ScanSums scan_sums(int64_t batch, int64_t seqlen, int64_t channels, int64_t dstate, int64_t ngroups, int gblocks) {
    ScanSums s;
    s.rates = channels * dstate;
    s.rows = gblocks == 1 ? 0 : batch * seqlen * ngroups * dstate;
    s.groups = (s.rates + 2 * channels + 2 * s.rows + kSumOutputs - 1) / kSumOutputs;
    s.blocks = (unsigned)(s.groups < (int64_t)1 << 20 ? s.groups : (int64_t)1 << 20);
    return s;
}

hipError_t launch_scan_fwd(const ScanArgs &a, const ScanPlan &plan, hipStream_t stream);
hipError_t launch_scan_bwd(const ScanArgs &a, const ScanPlan &plan, hipStream_t stream);
hipError_t launch_scan_step(const ScanArgs &a, hipStream_t stream);

}  // namespace ssd
