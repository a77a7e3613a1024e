// ks_scan.hip -- the selective scan's forward pass and its one-token step.
#include "ks_scan.h"

namespace ssd {
namespace {

// SUMMARY: a segment's own end state from a zero start, and the sum of its
// step sizes (whose exponential carries a state across the segment).
// Otherwise the outputs, from the segment's start state.
template <typename Tin, typename Tout, int LPC, bool SUMMARY>
__global__ __launch_bounds__(256) void ks_scan(ScanIn<Tin> a, const float *init, float *seg_state,
                                               float *__restrict__ seg_steps, Tout *__restrict__ y,
                                               float *final_state) {
    constexpr int NP = 4 * LPC, TPL = kTT / LPC;
    __shared__ float sB[2][kTT * NP], sC[2][SUMMARY ? 1 : kTT * NP];
    const ScanPos<LPC> at(a);
    const int n0 = 4 * at.j, b = at.b, c = at.c;
    const int64_t bc = (int64_t)b * a.channels + c;
    const int64_t slot = ((int64_t)b * a.nseg + at.seg) * a.channels + c;

    float A2[4], h[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        A2[r] = n0 + r < a.N ? rate(a.A[(int64_t)c * a.N + n0 + r]) : 0.f;
        h[r] = 0.f;
    }
    if (!SUMMARY) {
        if (a.nseg > 1) load_states(seg_state + slot * NP + n0, h);
        else load_states_n(init != nullptr ? init + bc * a.N : nullptr, n0, a.N, h);
    }
    const float bias = a.bias != nullptr ? a.bias[c] : 0.f;
    const float D = !SUMMARY && a.D != nullptr ? a.D[c] : 0.f;
    const bool gate = !SUMMARY && a.z != nullptr;
    float steps = 0.f;

    OwnRows<kTT, LPC, Tin> dts(a.dt, a.dts, b, c, at.j, at.ok, at.s0), xs(a.x, a.xs, b, c, at.j, at.ok, at.s0),
        zs(gate ? a.z : a.x, gate ? a.zs : a.xs, b, c, at.j, at.ok, at.s0);
    OwnRows<kTT, LPC, Tout> ys(y, Strides{(int64_t)a.L * a.channels, a.channels}, b, c, at.j, at.ok, at.s0);
    RowStage<kTT, NP, Tin> rB(a.B, a.Bs, b, at.g, a.N, at.s0), rC(a.C, a.Cs, b, at.g, a.N, at.s0);
    uint32_t dr[TPL], xr[TPL], zr[TPL];
    auto fetch = [&](int left) {
        dts.load(left, dr);
        xs.load(left, xr);
        if (gate) zs.load(left, zr);
        rB.load(left);
        if (!SUMMARY) rC.load(left);
        dts.next();
        xs.next();
        zs.next();
        rB.next();
        rC.next();
    };
    if (at.s0 < at.end) fetch(at.end - at.s0);
    int buf = 0, t = at.s0;
    for (; t < at.end; t += kTT, buf ^= 1) {
        const int left = at.end - t;
        rB.store(sB[buf]);
        if (!SUMMARY) rC.store(sC[buf]);
        float d[TPL], x[TPL], scale[TPL];
        step_sizes<kTT, LPC, Tin>(dr, bias, a.softplus, left, at.j, d);
#pragma unroll
        for (int i = 0; i < TPL; ++i) {
            x[i] = widen<Tin>(xr[i]);
            scale[i] = 1.f;
        }
        if (gate) {
#pragma unroll
            for (int i = 0; i < TPL; ++i) {
                const float z = widen<Tin>(zr[i]);
                scale[i] = z * logistic(z);
            }
        }
        __syncthreads();  // also: the buffer stored next was last read before this barrier
        if (left > kTT) fetch(left - kTT);
        float o[TPL];
#pragma unroll
        for (int i = 0; i < TPL; ++i) {
            const float u = taken(d[i]) * x[i];
            steps += d[i];
            float p[LPC];
            for_lanes<LPC>([&](auto K) {
                constexpr int k = decltype(K)::value;
                const float dk = lane_bcast<LPC, k>(d[i]), uk = lane_bcast<LPC, k>(u);
                const int row = (i * LPC + k) * NP + n0;
                const floatx4 Bv = *reinterpret_cast<const floatx4 *>(&sB[buf][row]);
#pragma unroll
                for (int r = 0; r < 4; ++r) h[r] = fmaf(fast_exp2(dk * A2[r]), h[r], uk * Bv[r]);
                if constexpr (!SUMMARY) {
                    const floatx4 Cv = *reinterpret_cast<const floatx4 *>(&sC[buf][row]);
                    float s = Cv[0] * h[0];
#pragma unroll
                    for (int r = 1; r < 4; ++r) s = fmaf(Cv[r], h[r], s);
                    p[k] = s;
                }
            });
            if constexpr (!SUMMARY) o[i] = fmaf(D, x[i], lane_sums<LPC>(p, at.j)) * scale[i];
        }
        if constexpr (!SUMMARY) {
            if (left < kTT) {
#pragma unroll
                for (int i = 0; i < TPL; ++i) o[i] = i * LPC + at.j < left ? o[i] : 0.f;
            }
            ys.store(at.s1 - t, o);
            ys.next();
        }
    }
    if constexpr (SUMMARY) {
        steps = lane_total<LPC>(steps);
        if (at.ok) {
            store_states(seg_state + slot * NP + n0, h);
            if (at.j == 0) seg_steps[slot] = steps;
        }
    } else {
        // tiles wholly behind the end
        const float zero[TPL] = {};
        for (; t < at.s1; t += kTT, ys.next()) ys.store(at.s1 - t, zero);
        if (at.seg == a.nseg - 1 && final_state != nullptr && at.ok)
            store_states_n(final_state + bc * a.N, n0, a.N, h);
    }
}

// The state at each segment's start, written over the segments' own end
// states: h <- exp(A sum of steps) h + own.  The last segment has no own end
// state: no segment starts from it.
__global__ __launch_bounds__(256) void ks_carry(const float *__restrict__ A, const float *__restrict__ init,
                                                float *__restrict__ seg_state, const float *__restrict__ seg_steps,
                                                int channels, int N, int NP, int nseg) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int b = blockIdx.y;
    if (i >= (int64_t)channels * NP) return;
    const int c = (int)(i / NP), n = (int)(i % NP);
    const bool ok = n < N;
    const float A2 = ok ? rate(A[(int64_t)c * N + n]) : 0.f;
    float *state = seg_state + (int64_t)b * nseg * channels * NP + i;
    const float h = carry_segments(ok && init != nullptr ? init[((int64_t)b * channels + c) * N + n] : 0.f, A2, state,
                                   seg_steps + (int64_t)b * nseg * channels + c, (int64_t)channels * NP, channels,
                                   nseg - 1, false);
    state[(int64_t)(nseg - 1) * channels * NP] = h;
}

// What one token of one channel brings beside its states.
template <typename Tin>
struct StepToken {
    float x, d, z, D;
    __device__ __forceinline__ StepToken(const ScanIn<Tin> &a, int b, int c) {
        x = load_one(a.x + b * a.xs.batch, c);
        const float raw = load_one(a.dt + b * a.dts.batch, c) + (a.bias != nullptr ? a.bias[c] : 0.f);
        z = a.z != nullptr ? load_one(a.z + b * a.zs.batch, c) : 0.f;
        D = a.D != nullptr ? a.D[c] : 0.f;
        d = held_step(a.softplus ? softplus(raw) : raw);
    }
    __device__ __forceinline__ float output(float s, bool gate) const {
        const float o = fmaf(D, x, s);
        return gate ? o * (z * logistic(z)) : o;
    }
};

// One token: a stream of the state (bound by memory, 8 bytes a state), a
// thread four neighbouring entries as one 16-byte piece (5120 channels of 16,
// batch 128: 5.2 TB/s, the rate of a copy).
// FULL: no lane without states (a branch around the loads costs 7 % there).
template <typename Tin, typename Tout, int LPC, bool FULL>
__global__ __launch_bounds__(256) void ks_step(ScanIn<Tin> a, float *state, Tout *__restrict__ y) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int b = blockIdx.y, n0 = 4 * (int)(i % LPC);
    if (i / LPC >= a.channels) return;  // whole channels: their lanes leave together
    const int c = (int)(i / LPC), g = c / a.cpg;
    const int64_t bc = (int64_t)b * a.channels + c;
    float h[4] = {}, A[4] = {}, Bv[4] = {}, Cv[4] = {};
    if (FULL || n0 < a.N) {
        load_states(state + bc * a.N + n0, h);
        load_states(a.A + (int64_t)c * a.N + n0, A);
        const Tin *Bp = a.B + b * a.Bs.batch + (int64_t)g * a.N, *Cp = a.C + b * a.Cs.batch + (int64_t)g * a.N;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            Bv[r] = load_one(Bp, n0 + r);
            Cv[r] = load_one(Cp, n0 + r);
        }
    }
    const StepToken<Tin> tok(a, b, c);
    const float u = taken(tok.d) * tok.x;
    float s = 0.f;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        h[r] = fmaf(fast_exp2(kLog2e * A[r] * tok.d), h[r], u * Bv[r]);
        s = fmaf(Cv[r], h[r], s);
    }
    if (FULL || n0 < a.N) store_states(state + bc * a.N + n0, h);
    s = lane_total<LPC>(s);
    if (n0 == 0) {
        const float o[1] = {tok.output(s, a.z != nullptr)};
        store_n<1>(y + bc, o);
    }
}

// The same for states of any number and alignment: a lane's entries lie LPC
// apart, so that the lanes of a channel read neighbouring words, and a thread
// takes the same entries of four channels, whose B and C it loads once (186 x
// 3075 channels of 35 states: 51 us against 103 us with four neighbouring
// entries of one channel a thread).
constexpr int kStepChannels = 4;
template <typename Tin, typename Tout, int LPC, int R>
__global__ __launch_bounds__(256) void ks_step_any(ScanIn<Tin> a, float *state, Tout *__restrict__ y) {
    constexpr int Q = kStepChannels, CB = 256 / LPC;
    const int b = blockIdx.y, j = threadIdx.x % LPC;
    const int first = blockIdx.x * CB * Q + threadIdx.x / LPC;  // then every CB-th channel
    float h[Q][R], A[Q][R], Bv[R], Cv[R];
    int held = -1;  // the group of Bv and Cv
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int c = first + q * CB;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int n = j + LPC * r;
            const bool in = c < a.channels && n < a.N;
            h[q][r] = in ? state[((int64_t)b * a.channels + c) * a.N + n] : 0.f;
            A[q][r] = in ? a.A[(int64_t)c * a.N + n] : 0.f;
        }
    }
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int c = first + q * CB;
        if (c >= a.channels) return;  // whole channels, and the later ones too
        const int g = c / a.cpg;
        if (g != held) {
            held = g;
            const Tin *Bp = a.B + b * a.Bs.batch + (int64_t)g * a.N, *Cp = a.C + b * a.Cs.batch + (int64_t)g * a.N;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int n = j + LPC * r;
                Bv[r] = n < a.N ? load_one(Bp, n) : 0.f;
                Cv[r] = n < a.N ? load_one(Cp, n) : 0.f;
            }
        }
        const int64_t bc = (int64_t)b * a.channels + c;
        const StepToken<Tin> tok(a, b, c);
        const float u = taken(tok.d) * tok.x;
        float s = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            h[q][r] = fmaf(fast_exp2(kLog2e * A[q][r] * tok.d), h[q][r], u * Bv[r]);
            s = fmaf(Cv[r], h[q][r], s);
            if (j + LPC * r < a.N) state[bc * a.N + j + LPC * r] = h[q][r];
        }
        s = lane_total<LPC>(s);
        if (j == 0) {
            const float o[1] = {tok.output(s, a.z != nullptr)};
            store_n<1>(y + bc, o);
        }
    }
}

template <typename Tin, typename Tout, int LPC>
hipError_t fwd(const ScanArgs &a, const ScanPlan &plan, hipStream_t stream) {
    const ScanIn<Tin> in = scan_in<Tin>(a, plan);
    const dim3 grid((unsigned)(plan.nblk * plan.nseg), (unsigned)a.batch);
    if (plan.nseg > 1) {
        const dim3 all_but_last((unsigned)(plan.nblk * (plan.nseg - 1)), (unsigned)a.batch);
        hipError_t e = launch_kernel(ks_scan<Tin, Tout, LPC, true>, all_but_last, dim3(256), 0, stream, LaunchEvents{},
                                     in, a.init, a.seg_state, a.seg_steps, (Tout *)nullptr, (float *)nullptr);
        if (e != hipSuccess) return e;
        const int64_t n = (int64_t)a.channels * plan.np;
        e = launch_kernel(ks_carry, dim3((unsigned)((n + 255) / 256), (unsigned)a.batch), dim3(256), 0, stream,
                          LaunchEvents{}, a.A, a.init, a.seg_state, (const float *)a.seg_steps, a.channels, a.dstate,
                          plan.np, plan.nseg);
        if (e != hipSuccess) return e;
    }
    return launch_kernel(ks_scan<Tin, Tout, LPC, false>, grid, dim3(256), 0, stream, LaunchEvents{}, in, a.init,
                         a.seg_state, a.seg_steps, static_cast<Tout *>(a.y), a.final_state);
}

template <typename Tin>
ScanIn<Tin> step_in(const ScanArgs &a) {
    ScanPlan plan{};
    plan.nblk = plan.gblocks = plan.nseg = 1;
    return scan_in<Tin>(a, plan);
}

template <typename Tin, typename Tout, int LPC>
hipError_t step(const ScanArgs &a, hipStream_t stream) {
    const dim3 grid((unsigned)(((int64_t)a.channels * LPC + 255) / 256), (unsigned)a.batch);
    const auto kernel = a.dstate == 4 * LPC ? ks_step<Tin, Tout, LPC, true> : ks_step<Tin, Tout, LPC, false>;
    return launch_kernel(kernel, grid, dim3(256), 0, stream, LaunchEvents{}, step_in<Tin>(a),
                         const_cast<float *>(a.init), static_cast<Tout *>(a.y));
}

template <typename Tin, typename Tout, int LPC, int R>
hipError_t step_any(const ScanArgs &a, hipStream_t stream) {
    const int cb = 256 / LPC * kStepChannels;
    const dim3 grid((unsigned)((a.channels + cb - 1) / cb), (unsigned)a.batch);
    return launch_kernel(ks_step_any<Tin, Tout, LPC, R>, grid, dim3(256), 0, stream, LaunchEvents{}, step_in<Tin>(a),
                         const_cast<float *>(a.init), static_cast<Tout *>(a.y));
}

template <typename Tin, typename Tout>
hipError_t fwd_np(const ScanArgs &a, const ScanPlan &plan, hipStream_t s) {
    switch (plan.np) {
        case 8: return fwd<Tin, Tout, 2>(a, plan, s);
        case 16: return fwd<Tin, Tout, 4>(a, plan, s);
        case 32: return fwd<Tin, Tout, 8>(a, plan, s);
        case 64: return fwd<Tin, Tout, 16>(a, plan, s);
        default: return hipErrorInvalidValue;
    }
}

// 16-byte pieces where every channel's states are whole ones
template <typename Tin, typename Tout>
hipError_t step_n(const ScanArgs &a, hipStream_t s) {
    const int n = a.dstate;
    if (n % 4 == 0 && (uintptr_t)a.init % 16 == 0 && (uintptr_t)a.A % 16 == 0) {
        switch (padded_states(n)) {
            case 8: return step<Tin, Tout, 2>(a, s);
            case 16: return step<Tin, Tout, 4>(a, s);
            case 32: return step<Tin, Tout, 8>(a, s);
            default: return step<Tin, Tout, 16>(a, s);
        }
    }
    if (n <= 8) return step_any<Tin, Tout, 8, 1>(a, s);
    if (n <= 16) return step_any<Tin, Tout, 16, 1>(a, s);
    if (n <= 32) return step_any<Tin, Tout, 16, 2>(a, s);
    if (n <= 48) return step_any<Tin, Tout, 16, 3>(a, s);
    return step_any<Tin, Tout, 16, 4>(a, s);
}

}  // namespace

hipError_t launch_scan_fwd(const ScanArgs &a, const ScanPlan &plan, hipStream_t s) {
    if (!a.in_bf16) return fwd_np<float, float>(a, plan, s);
    return a.y_bf16 ? fwd_np<uint16_t, uint16_t>(a, plan, s) : fwd_np<uint16_t, float>(a, plan, s);
}

hipError_t launch_scan_step(const ScanArgs &a, hipStream_t s) {
    if (!a.in_bf16) return step_n<float, float>(a, s);
    return a.y_bf16 ? step_n<uint16_t, uint16_t>(a, s) : step_n<uint16_t, float>(a, s);
}

}  // namespace ssd
