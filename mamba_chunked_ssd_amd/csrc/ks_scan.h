// ks_scan.h -- what the selective scan's kernels share (ks_scan.hip,
// ks_scan_bwd.hip).
//
//   d_t = softplus(dt_t + bias) ,  h_t = exp(d_t A) h_{t-1} + d_t x_t B_t ,
//   y_t = (C_t . h_t + D x_t) silu(z_t)
//
// for every channel and each of its states.  Unlike the chunked scan's, the
// decay belongs to (token, channel, state), so no product of matrices shares
// it: each state costs a product, an exponential (two issue slots), the input's
// product and two fused multiply-adds per token, and the scan is bound by
// vector instructions, not by memory.  2 x 2048 tokens of 5120 channels and 16
// states, bf16: six slots a state are 53 us at the measured 4.17 cycles a slot
// on 1024 SIMDs; the output pass takes 91 (9 slots a state, VALUBusy 90 %), the
// summary pass before it 67; their bytes at a copy's rate 32.
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

constexpr int kTT = 16;  // tokens of one tile (the backward pass's main kernel: kScanTile)

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
    int j, cl, c, c0, g, b, seg, blk;  // c0: the block's first channel
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
        c0 = g * a.cpg + (blk % a.gblocks) * CB;
        c = g * a.cpg + (ok ? in_group : 0);
        const int len = a.lengths == nullptr ? a.L : min(max(a.lengths[b], 0), a.L);
        s0 = min(seg * a.seglen, a.L);
        s1 = min(s0 + a.seglen, a.L);
        end = min(s1, len);
    }
};

// Rows of one sequence seen from a tile of TT tokens: a raw buffer over the
// tile's rows up to the segment's end, so that rows behind it read 0 and their
// stores are dropped without a branch.  Offsets into the tile are 32-bit (the
// entry points refuse row strides of 2^24 elements or more) and the same for
// every tile; the scalar unit moves the base from tile to tile.
template <int TT, typename T, bool FORTH = true>
struct TileRows {
    const T *at;   // the tile's first row
    uint32_t row;  // bytes of a row (a tile's are below 2^30: one scalar register each, of which the streams take many)
    __device__ __forceinline__ TileRows(const T *p, const Strides &s, int b, int t)
        : at(p + b * s.batch + t * s.row), row((uint32_t)(s.row * (int64_t)sizeof(T))) {}
    __device__ __forceinline__ void next() {
        const int64_t move = (uint32_t)TT * row;
        at = reinterpret_cast<const T *>(reinterpret_cast<uintptr_t>(at) + (FORTH ? move : -move));
    }
    // left: rows from the tile's first to the end
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t tile(int left) const {
        return uniform_rsrc(at, (uint32_t)min(max(left, 0), TT) * row);
    }
    __device__ __forceinline__ uint32_t offset(int token, int column) const {
        return token * row + column * (uint32_t)sizeof(T);
    }
};

// Loaded bits are widened only where they are used: a shift beside the load
// would wait for it, and the loads of the next tile are to be in flight over
// this one's work.
__device__ __forceinline__ uint32_t raw_load(const float *, __amdgpu_buffer_rsrc_t r, uint32_t off) {
    return __builtin_amdgcn_raw_buffer_load_b32(r, (int)off, 0, 0);
}
__device__ __forceinline__ uint32_t raw_load(const uint16_t *, __amdgpu_buffer_rsrc_t r, uint32_t off) {
    return (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, (int)off, 0, 0);
}
template <typename T>
__device__ __forceinline__ float widen(uint32_t bits) {
    return sizeof(T) == 2 ? bf16_to_f32(bits) : __uint_as_float(bits);
}
__device__ __forceinline__ void raw_store(float *, __amdgpu_buffer_rsrc_t r, uint32_t off, float v) {
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), r, (int)off, 0, 0);
}
__device__ __forceinline__ void raw_store(uint16_t *, __amdgpu_buffer_rsrc_t r, uint32_t off, float v) {
    __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(pack_bf16(v, 0.f) & 0xffffu), r, (int)off, 0, 0);
}

// A lane's own tokens of a tile, i LPC + j, of one channel: one offset, and a
// uniform step between the tokens.  HOLD keeps the offsets in registers over
// the tiles; without, they are formed again at every tile.  Where a tile has
// fewer tokens than a channel lanes, the lanes behind own none.
template <int TT, int LPC>
constexpr int own_tokens() { return TT >= LPC ? TT / LPC : 1; }
template <int TT, int LPC, typename T, bool HOLD = true, bool FORTH = true>
struct OwnRows {
    static constexpr int TPL = own_tokens<TT, LPC>();
    TileRows<TT, T, FORTH> rows;
    uint32_t first;
    __device__ __forceinline__ OwnRows(const T *p, const Strides &s, int b, int c, int j, bool ok, int t)
        : rows(p, s, b, t), first(ok && j < TT ? rows.offset(j, c) : kNowhere) {}
    __device__ __forceinline__ void next() { rows.next(); }
    __device__ __forceinline__ uint32_t base() const {
        uint32_t o = first;
        if constexpr (!HOLD) asm volatile("" : "+v"(o));
        return o;
    }
    __device__ __forceinline__ void load(int left, uint32_t (&v)[TPL]) const {
        const __amdgpu_buffer_rsrc_t r = rows.tile(left);
        const uint32_t o = base();
#pragma unroll
        for (int i = 0; i < TPL; ++i) v[i] = raw_load((const T *)nullptr, r, o + i * LPC * rows.row);
    }
    __device__ __forceinline__ void store(int left, const float (&v)[TPL]) const {
        const __amdgpu_buffer_rsrc_t r = rows.tile(left);
        const uint32_t o = base();
#pragma unroll
        for (int i = 0; i < TPL; ++i) raw_store((T *)nullptr, r, o + i * LPC * rows.row, v[i]);
    }
};

// One element of B or C per thread and tile: the group's rows, padded states
// and tokens behind the end as 0.
template <int TT, int NP, typename T, bool FORTH = true>
struct RowStage {
    static constexpr int E = (TT * NP + 255) / 256;
    TileRows<TT, T, FORTH> rows;
    uint32_t off[E], v[E];
    __device__ __forceinline__ RowStage(const T *p, const Strides &s, int b, int g, int N, int t) : rows(p, s, b, t) {
#pragma unroll
        for (int k = 0; k < E; ++k) {
            const int e = threadIdx.x + 256 * k, tok = e / NP, n = e % NP;
            off[k] = e < TT * NP && n < N ? rows.offset(tok, g * N + n) : kNowhere;
        }
    }
    __device__ __forceinline__ void next() { rows.next(); }
    __device__ __forceinline__ void load(int left) {
        const __amdgpu_buffer_rsrc_t r = rows.tile(left);
#pragma unroll
        for (int k = 0; k < E; ++k) v[k] = raw_load((const T *)nullptr, r, off[k]);
    }
    __device__ __forceinline__ void store(float *lds) const {
#pragma unroll
        for (int k = 0; k < E; ++k) {
            const int e = threadIdx.x + 256 * k;
            if (TT * NP >= 256 * (k + 1) || e < TT * NP) lds[e] = widen<T>(v[k]);
        }
    }
};

// A token's step size as its decay takes it: never 0, which an infinite rate
// would leave undefined (0 times infinity) where it is to keep nothing.  What is
// added changes no step of 2^-96 or more, and brings the exponent to -256 at
// that rate and to 0 at any below 2^95; other products take the step without it.
constexpr float kLeastStep = 0x1p-120f;
__device__ __forceinline__ float held_step(float d) { return d + kLeastStep; }
__device__ __forceinline__ float taken(float held) { return held - kLeastStep; }

// Step sizes of a lane's own tokens; rows behind the end take a step of 0, so
// the state stays.
template <int TT, int LPC, typename T>
__device__ __forceinline__ void step_sizes(const uint32_t (&dt)[own_tokens<TT, LPC>()], float bias, bool sp, int left, int j,
                                           float (&d)[own_tokens<TT, LPC>()]) {
    constexpr int TPL = own_tokens<TT, LPC>();
#pragma unroll
    for (int i = 0; i < TPL; ++i) d[i] = widen<T>(dt[i]) + bias;
    if (sp) {
#pragma unroll
        for (int i = 0; i < TPL; ++i) d[i] = softplus(d[i]);
    }
#pragma unroll
    for (int i = 0; i < TPL; ++i) d[i] = held_step(d[i]);
    if (left < TT) {
#pragma unroll
        for (int i = 0; i < TPL; ++i) d[i] = i * LPC + j < left ? d[i] : 0.f;
    }
}

// p[t] of a tile's tokens summed over a channel's lanes: v[i] for a lane's own
// token i LPC + j.
template <int TT, int LPC>
__device__ __forceinline__ float own_sum(const float (&p)[TT], int i, int j) {
    if constexpr (TT >= LPC) {
        float v[LPC];
#pragma unroll
        for (int k = 0; k < LPC; ++k) v[k] = p[i * LPC + k];
        return lane_sums<LPC>(v, j);
    } else {
        static_assert(LPC == 2 * TT && LPC == 16, "two lanes a token");
        float v[TT];
#pragma unroll
        for (int k = 0; k < TT; ++k) v[k] = p[k] + lane_swap<8>(p[k]);
        return lane_sums<TT>(v, j % TT);
    }
}

// A block's padded states and one number per channel, of a row of channels
// kept in the workspace (16 bytes a thread): raw buffers again, from the
// block's first channel on.
template <int LPC>
struct BlockRows {
    uint32_t states, number;  // offsets; kNowhere for lanes without a channel
    __device__ __forceinline__ BlockRows(bool ok, int j, int cl)
        : states(ok ? 16 * threadIdx.x : kNowhere), number(ok ? 4 * cl : kNowhere) {}
    static __device__ __forceinline__ __amdgpu_buffer_rsrc_t of(const float *first, int elements) {
        return uniform_rsrc(first, 4 * elements);
    }
    __device__ __forceinline__ void load(const float *first, float (&h)[4]) const {
        const u32x4 v = buffer_load_x4(of(first, 1024), (int)states);
#pragma unroll
        for (int r = 0; r < 4; ++r) h[r] = __uint_as_float(v[r]);
    }
    __device__ __forceinline__ void store(float *first, const float (&h)[4]) const {
        u32x4 v;
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = __float_as_uint(h[r]);
        __builtin_amdgcn_raw_buffer_store_b128(v, of(first, 1024), (int)states, 0, 0);
    }
    __device__ __forceinline__ float load_number(const float *first) const {
        return buffer_load_f32(of(first, 256 / LPC), (int)number);
    }
    // by every lane of the channel alike
    __device__ __forceinline__ void store_number(float *first, float v) const {
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), of(first, 256 / LPC), (int)number, 0, 0);
    }
};

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

// The decay's rate in base 2, exp(d A) = exp2(d rate(A)), held finite: rows
// behind an end take steps of 0, and 0 times the infinite A of a state that
// keeps nothing would be NaN.  (The one-token step has no such rows and takes A
// as it is.)  A NaN stays one.
__device__ __forceinline__ float rate(float A) {
    constexpr float most = __FLT_MAX__;
    const float v = kLog2e * A;
    return v < -most ? -most : v > most ? most : v;
}

// One state of one channel over the segments, in their order (or backwards,
// for the gradient): each slot's own end value gives way to the value it
// starts from, h <- exp2(A2 sum of steps) h + own.  Eight slots are loaded
// before the first is overwritten, or every load would wait for the store
// before it.
__device__ __forceinline__ float carry_segments(float h, float A2, float *state, const float *steps, int64_t state_stride,
                                                int64_t steps_stride, int nseg, bool backwards) {
    constexpr int G = 8;
    for (int q = 0; q < nseg; q += G) {
        float own[G], d[G];
#pragma unroll
        for (int e = 0; e < G; ++e) {
            const int k = backwards ? nseg - 1 - q - e : q + e;
            own[e] = q + e < nseg ? state[k * state_stride] : 0.f;
            d[e] = q + e < nseg ? steps[k * steps_stride] : 0.f;
        }
#pragma unroll
        for (int e = 0; e < G; ++e) {
            const int k = backwards ? nseg - 1 - q - e : q + e;
            if (q + e < nseg) {
                state[k * state_stride] = h;
                h = fmaf(fast_exp2(A2 * d[e]), h, own[e]);
            }
        }
    }
    return h;
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
