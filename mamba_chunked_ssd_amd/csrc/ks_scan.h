// ks_scan.h -- what the selective scan's kernels share (ks_scan.hip,
// ks_scan_bwd.hip).
//
//   d_t = softplus(dt_t + bias) ,  h_t = exp(d_t A) h_{t-1} + d_t x_t B_t ,
//   y_t = (C_t . h_t + D x_t) silu(z_t)
//
// for every channel and each of its states.  Unlike the chunked scan's, the
// decay belongs to (token, channel, state), so no product of matrices shares
// it: each state costs a product, an exponential (a quarter-rate instruction),
// the input's product and two fused multiply-adds per token, and the scan is
// bound by vector instructions, not by memory (16 states: about 190 issue
// cycles a lane for each token of a channel against 8 bytes).
//
// Layout: a channel's NP padded states lie on LPC = NP / 4 neighbouring lanes,
// four states a lane in registers, walking the tokens in order.  B_t and C_t,
// shared by all channels of a group, are staged in LDS as fp32 (one 16-byte
// read per lane and token); what is one number per (token, channel) -- the
// softplus, the gate, the skip, loads and stores -- is done once, by the lane
// whose turn the token is (token i LPC + j by lane j), and reaches the others
// by DPP broadcasts; the sum over states that crosses lanes is taken for LPC
// tokens at a time (lane_sums), each lane ending with its own token's.
#pragma once

#include "ssd_launch.h"
#include "ssd_ops_device.h"
#include "ssd_ops_internal.h"

namespace ssd {

constexpr int kTT = kScanTile;  // tokens of one tile

// Kernel arguments with typed inputs.
template <typename T>
struct ScanIn {
    const T *x, *dt, *B, *C, *z;
    const float *A, *D, *bias;
    const int32_t *lengths;
    Strides xs, dts, Bs, Cs, zs;
    int L, channels, N, cpg;          // cpg: channels of a group
    int nblk, gblocks, nseg, seglen;  // ScanPlan
    bool softplus;
};

// Where a thread stands: its channel, its lane j of the channel's LPC, its
// segment and how far the sequence reaches into it.
template <int LPC>
struct ScanPos {
    static constexpr int NP = 4 * LPC;
    static constexpr int CB = 256 / LPC;  // channels of a block
    int j, cl, c, g, b, seg, blk;
    bool ok;     // c exists (else it stands in for the group's first)
    int s0, s1;  // the segment's tokens
    int end;     // of them, those before `end` belong to the sequence

    template <typename T>
    __device__ __forceinline__ ScanPos(const ScanIn<T> &a) {
        const int tid = threadIdx.x;
        j = tid % LPC;
        cl = tid / LPC;
        blk = blockIdx.x % a.nblk;
        seg = blockIdx.x / a.nblk;
        b = blockIdx.y;
        g = blk / a.gblocks;
        const int in_group = (blk % a.gblocks) * CB + cl;
        ok = in_group < a.cpg;
        c = g * a.cpg + (ok ? in_group : 0);
        const int len = a.lengths == nullptr ? a.L : min(max(a.lengths[b], 0), a.L);
        s0 = min(seg * a.seglen, a.L);
        s1 = min(s0 + a.seglen, a.L);
        end = min(s1, len);
    }
};

// One element of B or C per thread and tile: rows t .. t + kTT - 1 of the
// group, padded states and tokens behind the end as 0.
template <int NP, typename T>
struct RowStage {
    static constexpr int E = (kTT * NP + 255) / 256;
    float v[E];
    __device__ __forceinline__ void load(const T *p, const Strides &st, int b, int g, int N, int t, int end) {
#pragma unroll
        for (int k = 0; k < E; ++k) {
            const int e = threadIdx.x + 256 * k, tok = e / NP, n = e % NP;
            v[k] = e < kTT * NP && n < N && t + tok < end && t + tok >= 0
                       ? load_one(p + b * st.batch + (t + tok) * st.row + (int64_t)g * N, n)
                       : 0.f;
        }
    }
    __device__ __forceinline__ void store(float *lds) const {
#pragma unroll
        for (int k = 0; k < E; ++k) {
            const int e = threadIdx.x + 256 * k;
            if (e < kTT * NP) lds[e] = v[k];
        }
    }
};

// The values of a lane's own tokens of a tile, t + i LPC + j.
template <int LPC, typename T>
__device__ __forceinline__ void load_own(const T *p, const Strides &st, int b, int c, int t, int j, int end,
                                         float (&v)[kTT / LPC]) {
#pragma unroll
    for (int i = 0; i < kTT / LPC; ++i) {
        const int tt = t + i * LPC + j;
        v[i] = tt < end ? load_one(p + b * st.batch + tt * st.row, c) : 0.f;
    }
}

// Four states of (row, channel) in padded fp32 storage.
__device__ __forceinline__ void load_states(const float *p, float (&h)[4]) {
    const floatx4 v = *reinterpret_cast<const floatx4 *>(p);
#pragma unroll
    for (int r = 0; r < 4; ++r) h[r] = v[r];
}
__device__ __forceinline__ void store_states(float *p, const float (&h)[4]) {
    *reinterpret_cast<floatx4 *>(p) = floatx4{h[0], h[1], h[2], h[3]};
}
// The same from and to the caller's (batch, channels, N), N any size.
__device__ __forceinline__ void load_states_n(const float *p, int n0, int N, float (&h)[4]) {
#pragma unroll
    for (int r = 0; r < 4; ++r) h[r] = p != nullptr && n0 + r < N ? p[n0 + r] : 0.f;
}
__device__ __forceinline__ void store_states_n(float *p, int n0, int N, const float (&h)[4]) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
        if (n0 + r < N) p[n0 + r] = h[r];
}

template <typename T>
ScanIn<T> scan_in(const ScanArgs &a, const ScanPlan &plan) {
    ScanIn<T> in;
    in.x = static_cast<const T *>(a.x);
    in.dt = static_cast<const T *>(a.dt);
    in.B = static_cast<const T *>(a.B);
    in.C = static_cast<const T *>(a.C);
    in.z = static_cast<const T *>(a.z);
    in.A = a.A;
    in.D = a.D;
    in.bias = a.dt_bias;
    in.lengths = a.lengths;
    in.xs = a.xs;
    in.dts = a.dts;
    in.Bs = a.Bs;
    in.Cs = a.Cs;
    in.zs = a.zs;
    in.L = a.seqlen;
    in.channels = a.channels;
    in.N = a.dstate;
    in.cpg = a.channels / a.ngroups;
    in.nblk = plan.nblk;
    in.gblocks = plan.gblocks;
    in.nseg = plan.nseg;
    in.seglen = plan.seglen;
    in.softplus = a.softplus;
    return in;
}

}  // namespace ssd
