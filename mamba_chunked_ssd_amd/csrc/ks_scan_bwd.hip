// ks_scan_bwd.hip -- the selective scan's backward pass.
//
// With e_t = exp(d_t A) and o_t the gradient of the sum before the gate,
// backwards in t:
//   G_t = C_t o_t + e_{t+1} G_{t+1}                       (gradient of h_t)
//   dC_t = sum_c o_t h_t ,  dB_t = sum_c d_t x_t G_t       (over a group's channels)
//   q_t = e_t G_t h_{t-1}                                 (gradient of d_t A)
//   dA = sum_t d_t q_t ,  dd_t = sum_n A q_t + x_t sum_n B_t G_t
//   dx_t = d_t sum_n B_t G_t + D o_t ,  ddt_t = dd_t softplus'(dt_t + bias)
//   dz_t = dy_t (C_t . h_t + D x_t) silu'(z_t) ,  o_t = dy_t silu(z_t) .
//
// The states are not kept by the forward pass: one sweep stores the state
// before every tile of 16 tokens (as many bytes as one fp32 tensor of x's
// size), and the main kernel walks the tiles backwards, forming a tile's 16
// states and decays again in registers.  Bound by vector instructions, as the
// forward pass: about 30 issue slots per (token, channel, state) in all.
//
// dB and dC sum over channels, which lie across lanes.  That sum is left to
// the matrix cores, idle otherwise: v_mfma_f32_16x16x4_f32 with the values as
// A (row m = lane % 16, column k = lane / 16) and a column that is 1 for the
// token and 0 elsewhere as B adds the four channels of one k to column
// `token`, in fp32, so 16 tokens fill one accumulator; what is left (the
// channels that share rows, and the block's waves) is added once per tile
// from LDS.
#include "ks_scan.h"

namespace ssd {
namespace {

// The output's gradient before the gate, and what the gate's own needs.
__device__ __forceinline__ float ungate(float dy, float z, bool gate) { return gate ? dy * (z * logistic(z)) : dy; }

// One sweep over a segment.  SUMMARY: its own end state from a zero start, its
// own gradient at the start from a zero end, sum over t of
// (e_first .. e_t) C_t o_t, and the sum of its step sizes.  Otherwise the
// state before every tile, from the segment's start state.
template <typename Tin, typename Tdy, int LPC, bool SUMMARY>
__global__ __launch_bounds__(256) void ks_bwd_sweep(ScanIn<Tin> a, const Tdy *__restrict__ dy, Strides dys,
                                                    const float *__restrict__ init, float *__restrict__ seg_state,
                                                    float *__restrict__ seg_adj, float *__restrict__ seg_steps,
                                                    float *__restrict__ tile_state, int64_t tiles) {
    constexpr int NP = 4 * LPC, TPL = kTT / LPC;
    __shared__ float sB[2][kTT * NP], sC[2][SUMMARY ? kTT * NP : 1];
    const ScanPos<LPC> at(a);
    const int n0 = 4 * at.j, b = at.b, c = at.c;
    const int64_t slot = ((int64_t)b * a.nseg + at.seg) * a.channels + c;
    float A2[4], h[4], P[4], Gs[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        A2[r] = n0 + r < a.N ? kLog2e * a.A[(int64_t)c * a.N + n0 + r] : 0.f;
        h[r] = Gs[r] = 0.f;
        P[r] = 1.f;
    }
    if (!SUMMARY) {
        if (a.nseg > 1) load_states(seg_state + slot * NP + n0, h);
        else load_states_n(init != nullptr ? init + ((int64_t)b * a.channels + c) * a.N : nullptr, n0, a.N, h);
    }
    const float bias = a.bias != nullptr ? a.bias[c] : 0.f;
    const bool gate = SUMMARY && a.z != nullptr;
    float steps = 0.f;
    RowStage<NP, Tin> rB, rC;
    float dr[TPL], xr[TPL], zr[TPL], gr[TPL];
    auto fetch = [&](int t) {
        load_own<LPC>(a.dt, a.dts, b, c, t, at.j, at.end, dr);
        load_own<LPC>(a.x, a.xs, b, c, t, at.j, at.end, xr);
        rB.load(a.B, a.Bs, b, at.g, a.N, t, at.end);
        if constexpr (SUMMARY) {
            if (gate) load_own<LPC>(a.z, a.zs, b, c, t, at.j, at.end, zr);
            load_own<LPC>(dy, dys, b, c, t, at.j, at.end, gr);
            rC.load(a.C, a.Cs, b, at.g, a.N, t, at.end);
        }
    };
    if (at.s0 < at.end) fetch(at.s0);
    int buf = 0;
    for (int t = at.s0; t < at.end; t += kTT, buf ^= 1) {
        rB.store(sB[buf]);
        if constexpr (SUMMARY) rC.store(sC[buf]);
        else if (at.ok) store_states(tile_state + (((int64_t)b * tiles + t / kTT) * a.channels + c) * NP + n0, h);
        float d[TPL], u[TPL], o[TPL];
#pragma unroll
        for (int i = 0; i < TPL; ++i) {
            const float raw = dr[i] + bias;
            d[i] = t + i * LPC + at.j < at.end ? (a.softplus ? softplus(raw) : raw) : 0.f;
            u[i] = d[i] * xr[i];
            if constexpr (SUMMARY) o[i] = ungate(gr[i], zr[i], gate);
        }
        __syncthreads();
        if (t + kTT < at.end) fetch(t + kTT);
#pragma unroll
        for (int i = 0; i < TPL; ++i) {
            steps += d[i];
            for_lanes<LPC>([&](auto K) {
                constexpr int k = decltype(K)::value;
                const float dk = lane_bcast<LPC, k>(d[i]), uk = lane_bcast<LPC, k>(u[i]);
                const int row = (i * LPC + k) * NP + n0;
                const floatx4 Bv = *reinterpret_cast<const floatx4 *>(&sB[buf][row]);
                floatx4 Co;
                if constexpr (SUMMARY) {
                    const float ok = lane_bcast<LPC, k>(o[i]);
                    Co = *reinterpret_cast<const floatx4 *>(&sC[buf][row]) * ok;
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float e = fast_exp2(dk * A2[r]);
                    h[r] = fmaf(e, h[r], uk * Bv[r]);
                    if constexpr (SUMMARY) {
                        P[r] *= e;
                        Gs[r] = fmaf(P[r], Co[r], Gs[r]);
                    }
                }
            });
        }
    }
    if constexpr (SUMMARY) {
        steps = lane_total<LPC>(steps);
        if (at.ok) {
            store_states(seg_state + slot * NP + n0, h);
            store_states(seg_adj + slot * NP + n0, Gs);
            if (at.j == 0) seg_steps[slot] = steps;
        }
    }
}

// blockIdx.z 0: the state at each segment's start; 1: backwards, the gradient
// of the state at each segment's end, and of the initial state.
__global__ __launch_bounds__(256) void ks_bwd_carry(const float *__restrict__ A, const float *__restrict__ init,
                                                    const float *__restrict__ dfinal, float *__restrict__ seg_state,
                                                    float *__restrict__ seg_adj, const float *__restrict__ seg_steps,
                                                    float *__restrict__ dinit, int channels, int N, int NP, int nseg) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int b = blockIdx.y;
    if (i >= (int64_t)channels * NP) return;
    const bool adj = blockIdx.z != 0;
    const int c = (int)(i / NP), n = (int)(i % NP);
    const bool ok = n < N;
    const int64_t bcn = ((int64_t)b * channels + c) * N + n;
    const float A2 = ok ? kLog2e * A[(int64_t)c * N + n] : 0.f;
    const float *from = adj ? dfinal : init;
    float h = ok && from != nullptr ? from[bcn] : 0.f;
    float *s = (adj ? seg_adj : seg_state) + (int64_t)b * nseg * channels * NP + i;
    const float *sum = seg_steps + (int64_t)b * nseg * channels + c;
#pragma unroll 4
    for (int q = 0; q < nseg; ++q) {
        const int k = adj ? nseg - 1 - q : q;
        const float own = s[(int64_t)k * channels * NP], d = sum[(int64_t)k * channels];
        s[(int64_t)k * channels * NP] = h;
        h = fmaf(fast_exp2(A2 * d), h, own);
    }
    if (adj && ok && dinit != nullptr) dinit[bcn] = h;
}

struct BwdOut {
    float *dx, *ddt, *dz, *dinit;
    float *db, *dc;         // dB and dC, or a block's partial rows of them
    int64_t blk, tok;       // elements between blocks and between tokens there
    float *dap, *ddp, *dbiasp;
};

constexpr int kRedStride = kTT + 1;       // LDS row of 16 tokens, padded
constexpr int kRedWave = 64 * kRedStride;  // one wave's accumulator: 64 rows

template <typename Tin, typename Tdy, int LPC>
__global__ __launch_bounds__(256, 2) void ks_bwd_main(ScanIn<Tin> a, const Tdy *__restrict__ dy, Strides dys,
                                                      const float *__restrict__ dfinal,
                                                      const float *__restrict__ seg_adj,
                                                      const float *__restrict__ tile_state, int64_t tiles, BwdOut out) {
    constexpr int NP = 4 * LPC, TPL = kTT / LPC;
    __shared__ float sB[kTT * NP], sC[kTT * NP], red[2][4][kRedWave];
    const ScanPos<LPC> at(a);
    const int n0 = 4 * at.j, b = at.b, c = at.c;
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int64_t slot = ((int64_t)b * a.nseg + at.seg) * a.channels + c;
    const int64_t bc = (int64_t)b * a.channels + c;
    float A2[4], carry[4], dA[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        A2[r] = n0 + r < a.N ? kLog2e * a.A[(int64_t)c * a.N + n0 + r] : 0.f;
        dA[r] = 0.f;
    }
    if (a.nseg > 1) load_states(seg_adj + slot * NP + n0, carry);
    else load_states_n(dfinal != nullptr ? dfinal + bc * a.N : nullptr, n0, a.N, carry);
    const float bias = a.bias != nullptr ? a.bias[c] : 0.f;
    const float D = a.D != nullptr ? a.D[c] : 0.f;
    const bool gate = a.z != nullptr;
    float dD = 0.f, dbias = 0.f;

    // a block's last channels may stand in for the group's first: they add nothing to the sums over channels
    const float mine = at.ok ? 1.f : 0.f;
    float *db = out.db + at.blk * out.blk, *dc = out.dc + at.blk * out.blk;

    // rows behind the end
    const int done = at.end > at.s0 ? at.s0 + (at.end - at.s0 + kTT - 1) / kTT * kTT : at.s0;
    for (int tt = done + at.j; tt < at.s1; tt += LPC)
        if (at.ok) {
            const int64_t i = ((int64_t)b * a.L + tt) * a.channels + c;
            out.dx[i] = 0.f;
            out.ddt[i] = 0.f;
            if (gate) out.dz[i] = 0.f;
        }
    for (int64_t i = threadIdx.x; i < (int64_t)(at.s1 - done) * a.N; i += 256) {
        const int64_t p = ((int64_t)b * a.L + done + i / a.N) * out.tok + i % a.N;
        db[p] = 0.f;
        dc[p] = 0.f;
    }

    for (int t = done - kTT; t >= at.s0; t -= kTT) {
        RowStage<NP, Tin> rB, rC;
        float d[TPL], x[TPL], z[TPL], g[TPL], sl[TPL], o[TPL], dt[TPL];
        float h0[4];
        load_own<LPC>(a.dt, a.dts, b, c, t, at.j, at.end, dt);
        load_own<LPC>(a.x, a.xs, b, c, t, at.j, at.end, x);
        if (gate) load_own<LPC>(a.z, a.zs, b, c, t, at.j, at.end, z);
        load_own<LPC>(dy, dys, b, c, t, at.j, at.end, g);
        rB.load(a.B, a.Bs, b, at.g, a.N, t, at.end);
        rC.load(a.C, a.Cs, b, at.g, a.N, t, at.end);
        load_states(tile_state + (((int64_t)b * tiles + t / kTT) * a.channels + c) * NP + n0, h0);
        rB.store(sB);
        rC.store(sC);
        __syncthreads();

        float e[kTT][4], h[kTT][4], tot[TPL];
#pragma unroll
        for (int i = 0; i < TPL; ++i) {
            const bool live = t + i * LPC + at.j < at.end;
            const float raw = dt[i] + bias;
            d[i] = live ? (a.softplus ? softplus(raw) : raw) : 0.f;
            sl[i] = live ? (a.softplus ? logistic(raw) : 1.f) : 0.f;  // softplus', 0 behind the end
            o[i] = ungate(g[i], z[i], gate);
            const float u = d[i] * x[i];
            float p[LPC];
            for_lanes<LPC>([&](auto K) {
                constexpr int k = decltype(K)::value;
                const int tk = i * LPC + k;
                const float dk = lane_bcast<LPC, k>(d[i]), uk = lane_bcast<LPC, k>(u);
                const floatx4 Bv = *reinterpret_cast<const floatx4 *>(&sB[tk * NP + n0]);
                const floatx4 Cv = *reinterpret_cast<const floatx4 *>(&sC[tk * NP + n0]);
                p[k] = 0.f;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    e[tk][r] = fast_exp2(dk * A2[r]);
                    h[tk][r] = fmaf(e[tk][r], tk == 0 ? h0[r] : h[tk > 0 ? tk - 1 : 0][r], uk * Bv[r]);
                    p[k] = fmaf(Cv[r], h[tk][r], p[k]);
                }
            });
            tot[i] = lane_sums<LPC>(p, at.j);
        }

        floatx4 accB[4], accC[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) accB[r] = accC[r] = zero4();
#pragma unroll
        for (int ii = 0; ii < TPL; ++ii) {
            const int i = TPL - 1 - ii;
            const float u = d[i] * x[i];
            float pB[LPC], pA[LPC];
            for_lanes<LPC>([&](auto K) {
                constexpr int k = LPC - 1 - decltype(K)::value;
                const int tk = i * LPC + k;
                const float dk = lane_bcast<LPC, k>(d[i]), uk = lane_bcast<LPC, k>(u) * mine;
                const float ok = lane_bcast<LPC, k>(o[i]);
                const float om = ok * mine;
                const floatx4 Bv = *reinterpret_cast<const floatx4 *>(&sB[tk * NP + n0]);
                const floatx4 Cv = *reinterpret_cast<const floatx4 *>(&sC[tk * NP + n0]);
                const float column = lane % 16 == tk ? 1.f : 0.f;
                pB[k] = pA[k] = 0.f;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float G = fmaf(Cv[r], ok, carry[r]);
                    accC[r] = mfma_f32(om * h[tk][r], column, accC[r]);
                    accB[r] = mfma_f32(uk * G, column, accB[r]);
                    pB[k] = fmaf(G, Bv[r], pB[k]);
                    carry[r] = e[tk][r] * G;
                    const float q = carry[r] * (tk == 0 ? h0[r] : h[tk > 0 ? tk - 1 : 0][r]);
                    pA[k] = fmaf(q, A2[r], pA[k]);
                    dA[r] = fmaf(q, dk, dA[r]);
                }
            });
            const float gB = lane_sums<LPC>(pB, at.j), gA = lane_sums<LPC>(pA, at.j);
            const int tt = t + i * LPC + at.j;
            // pA used log2(e) A
            const float ddt = fmaf(0.6931471805599453f, gA, gB * x[i]) * sl[i];
            dbias += ddt;
            dD = fmaf(o[i], x[i], dD);
            if (at.ok && tt < at.s1) {
                const int64_t w = ((int64_t)b * a.L + tt) * a.channels + c;
                out.dx[w] = fmaf(gB, d[i], D * o[i]);
                out.ddt[w] = ddt;
                if (gate) {
                    const float s = logistic(z[i]);
                    out.dz[w] = g[i] * fmaf(D, x[i], tot[i]) * (s * fmaf(z[i], 1.f - s, 1.f));
                }
            }
        }

        // accumulator rows m = 4 (lane / 16) + q, columns the tokens; row (m, r) of the LDS tile is channel
        // m / LPC of its k and state 4 (m % LPC) + r
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int row = (4 * (lane / 16) + q) * 4 + r;
                red[0][wave][row * kRedStride + lane % 16] = accB[r][q];
                red[1][wave][row * kRedStride + lane % 16] = accC[r][q];
            }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * kTT * NP; i += 256) {
            const int n = i % NP, tok = i / NP % kTT, kind = i / (NP * kTT);
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < 4; ++w)
#pragma unroll
                for (int q = 0; q < 16 / LPC; ++q) s += red[kind][w][(q * NP + n) * kRedStride + tok];
            if (n < a.N && t + tok < at.s1) {
                const int64_t p = ((int64_t)b * a.L + t + tok) * out.tok + n;
                (kind == 0 ? db : dc)[p] = s;
            }
        }
    }

    if (at.ok) store_states(out.dap + slot * NP + n0, dA);
    dD = lane_total<LPC>(dD);
    dbias = lane_total<LPC>(dbias);
    if (at.ok && at.j == 0) {
        out.ddp[slot] = dD;
        out.dbiasp[slot] = dbias;
    }
    if (a.nseg == 1 && out.dinit != nullptr && at.ok) store_states_n(out.dinit + bc * a.N, n0, a.N, carry);
}

// The last sums, in a fixed order and 64 bits: dA, dD and ddt_bias over batch
// and segments; dB and dC over the blocks of each group (gblocks 1: written
// in place already).
struct BwdSums {
    const float *dap, *ddp, *dbiasp, *dbp, *dcp;
    float *dA, *dD, *ddt_bias, *dB, *dC;
    int64_t slots;        // batch * nseg
    int64_t rows;         // batch * seqlen
    int channels, N, NP, ngroups, gblocks;
};
__global__ __launch_bounds__(256) void ks_bwd_sums(BwdSums s, int64_t nA, int64_t nBC) {
    int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < nA) {
        const int64_t c = i / s.N, n = i % s.N;
        double v = 0.0;
        for (int64_t k = 0; k < s.slots; ++k) v += (double)s.dap[(k * s.channels + c) * s.NP + n];
        s.dA[i] = (float)v;
        return;
    }
    i -= nA;
    if (i < 2 * (int64_t)s.channels) {
        const bool first = i < s.channels;
        const int64_t c = first ? i : i - s.channels;
        float *to = first ? s.dD : s.ddt_bias;
        if (to == nullptr) return;
        const float *from = first ? s.ddp : s.dbiasp;
        double v = 0.0;
        for (int64_t k = 0; k < s.slots; ++k) v += (double)from[k * s.channels + c];
        to[c] = (float)v;
        return;
    }
    i -= 2 * (int64_t)s.channels;
    if (i >= 2 * nBC) return;
    const bool first = i < nBC;
    if (!first) i -= nBC;
    const int64_t n = i % s.N, g = i / s.N % s.ngroups, row = i / ((int64_t)s.N * s.ngroups);
    const float *from = (first ? s.dbp : s.dcp) + (g * s.gblocks * s.rows + row) * s.N + n;
    double v = 0.0;
    for (int k = 0; k < s.gblocks; ++k) v += (double)from[(int64_t)k * s.rows * s.N];
    (first ? s.dB : s.dC)[i] = (float)v;
}

template <typename Tin, typename Tdy, int LPC>
hipError_t bwd(const ScanArgs &a, const ScanPlan &plan, hipStream_t stream) {
    const ScanIn<Tin> in = scan_in<Tin>(a, plan);
    const Tdy *dy = static_cast<const Tdy *>(a.dy);
    const dim3 grid((unsigned)(plan.nblk * plan.nseg), (unsigned)a.batch);
    hipError_t e = hipSuccess;
    if (a.batch > 0) {
        if (plan.nseg > 1) {
            e = launch_kernel(ks_bwd_sweep<Tin, Tdy, LPC, true>, grid, dim3(256), 0, stream, LaunchEvents{}, in, dy,
                              a.dys, a.init, a.seg_state, a.seg_adj, a.seg_steps, a.tile_state, plan.tiles);
            if (e != hipSuccess) return e;
            const int64_t n = (int64_t)a.channels * plan.np;
            e = launch_kernel(ks_bwd_carry, dim3((unsigned)((n + 255) / 256), (unsigned)a.batch, 2), dim3(256), 0,
                              stream, LaunchEvents{}, a.A, a.init, a.dfinal, a.seg_state, a.seg_adj,
                              (const float *)a.seg_steps, a.dinit, a.channels, a.dstate, plan.np, plan.nseg);
            if (e != hipSuccess) return e;
        }
        if (a.seqlen > 0) {
            e = launch_kernel(ks_bwd_sweep<Tin, Tdy, LPC, false>, grid, dim3(256), 0, stream, LaunchEvents{}, in, dy,
                              a.dys, a.init, a.seg_state, a.seg_adj, a.seg_steps, a.tile_state, plan.tiles);
            if (e != hipSuccess) return e;
        }
        BwdOut out{a.dx, a.ddt, a.dz, a.dinit, a.dbp, a.dcp, a.batch * a.seqlen * a.dstate, a.dstate,
                   a.dap, a.ddp, a.dbiasp};
        if (plan.gblocks == 1) {  // one block a group: its rows are the outputs'
            out.db = a.dB;
            out.dc = a.dC;
            out.blk = a.dstate;
            out.tok = (int64_t)a.ngroups * a.dstate;
        }
        e = launch_kernel(ks_bwd_main<Tin, Tdy, LPC>, grid, dim3(256), 0, stream, LaunchEvents{}, in, dy, a.dys,
                          a.dfinal, (const float *)a.seg_adj, (const float *)a.tile_state, plan.tiles, out);
        if (e != hipSuccess) return e;
    }
    const BwdSums s{a.dap, a.ddp, a.dbiasp, a.dbp, a.dcp, a.dA, a.dD, a.ddt_bias, a.dB, a.dC,
                    a.batch * plan.nseg, a.batch * a.seqlen, a.channels, a.dstate, plan.np, a.ngroups, plan.gblocks};
    const int64_t nA = (int64_t)a.channels * a.dstate;
    const int64_t nBC = plan.gblocks == 1 ? 0 : a.batch * a.seqlen * a.ngroups * a.dstate;
    const int64_t n = nA + 2 * (int64_t)a.channels + 2 * nBC;
    return launch_kernel(ks_bwd_sums, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, stream, LaunchEvents{}, s, nA,
                         nBC);
}

template <typename Tin, typename Tdy>
hipError_t bwd_np(const ScanArgs &a, const ScanPlan &plan, hipStream_t s) {
    switch (plan.np) {
        case 8: return bwd<Tin, Tdy, 2>(a, plan, s);
        case 16: return bwd<Tin, Tdy, 4>(a, plan, s);
        case 32: return bwd<Tin, Tdy, 8>(a, plan, s);
        case 64: return bwd<Tin, Tdy, 16>(a, plan, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_scan_bwd(const ScanArgs &a, const ScanPlan &plan, hipStream_t s) {
    if (!a.in_bf16) return bwd_np<float, float>(a, plan, s);
    return a.y_bf16 ? bwd_np<uint16_t, uint16_t>(a, plan, s) : bwd_np<uint16_t, float>(a, plan, s);
}

}  // namespace ssd
