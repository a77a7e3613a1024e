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
// before every tile of 8 tokens (at 16 states as many bytes as two fp32 tensors
// of x's size), and the main kernel walks the tiles backwards, forming a tile's
// states and decays again in registers.  Where time is cut into segments the
// sweep runs each from a zero state, leaving local tile states, the segment's
// summary and its adjoint's together; the main kernel adds to a tile's local
// state what the segment's start state has become by then (one exponential a
// state and tile).  Bound by vector instructions, as the forward pass: 11
// issue slots per (token, channel, state) in the sweep, 26 in the main kernel (2 x
// 2048 tokens of 5120 channels and 16 states: sweep 132 us at VALUBusy 77 %,
// main kernel 296 at 74 %, carry 14, sums 17).
//
// dB and dC sum over channels, which lie across lanes and blocks: within a wave
// by channel_sums, the rest of the block once per tile from LDS, and the
// blocks' partial rows in ks_bwd_sums.
#include "ks_scan.h"

namespace ssd {
namespace {

// One sweep over a segment, storing the state before every tile.  SEGS (more
// than one segment): the states are those from a zero start, and with each
// goes the sum of the segment's steps before it; at the end the segment's own
// end state, its own gradient at the start from a zero end,
// sum over t of (e_first .. e_t) C_t o_t, and the sum of its steps.
template <typename Tin, typename Tdy, int LPC, bool SEGS>
__global__ __launch_bounds__(256) void ks_bwd_sweep(ScanIn<Tin> a, const Tdy *__restrict__ dy, Strides dys,
                                                    const float *__restrict__ init, float *__restrict__ seg_state,
                                                    float *__restrict__ seg_adj, float *__restrict__ seg_steps,
                                                    float *__restrict__ tile_state, float *__restrict__ tile_steps,
                                                    int64_t tiles) {
    constexpr int NP = 4 * LPC, TPL = kTT / LPC;
    __shared__ float sB[2][kTT * NP], sC[2][SEGS ? kTT * NP : 1];
    const ScanPos<LPC> at(a);
    const int n0 = 4 * at.j, b = at.b, c = at.c;
    const int64_t slot = ((int64_t)b * a.nseg + at.seg) * a.channels + c;
    float A2[4], h[4], P[4], Gs[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        A2[r] = n0 + r < a.N ? rate(a.A[(int64_t)c * a.N + n0 + r]) : 0.f;
        h[r] = Gs[r] = 0.f;
        P[r] = 1.f;
    }
    if (!SEGS) load_states_n(init != nullptr ? init + ((int64_t)b * a.channels + c) * a.N : nullptr, n0, a.N, h);
    const float bias = a.bias != nullptr ? a.bias[c] : 0.f;
    const bool gate = SEGS && a.z != nullptr;
    float steps = 0.f;
    OwnRows<kTT, LPC, Tin> dts(a.dt, a.dts, b, c, at.j, at.ok, at.s0), xs(a.x, a.xs, b, c, at.j, at.ok, at.s0),
        zs(gate ? a.z : a.x, gate ? a.zs : a.xs, b, c, at.j, at.ok, at.s0);
    OwnRows<kTT, LPC, Tdy> gs(dy, dys, b, c, at.j, at.ok, at.s0);
    RowStage<kTT, NP, Tin> rB(a.B, a.Bs, b, at.g, a.N, at.s0), rC(a.C, a.Cs, b, at.g, a.N, at.s0);
    uint32_t dr[TPL], xr[TPL], zr[TPL], gr[TPL];
    auto fetch = [&](int left) {
        dts.load(left, dr);
        xs.load(left, xr);
        rB.load(left);
        dts.next();
        xs.next();
        rB.next();
        if constexpr (SEGS) {
            if (gate) zs.load(left, zr);
            gs.load(left, gr);
            rC.load(left);
            zs.next();
            gs.next();
            rC.next();
        }
    };
    if (at.s0 < at.end) fetch(at.end - at.s0);
    int buf = 0;
    const BlockRows<LPC> mine(at.ok, at.j, at.cl);
    int64_t tile = ((int64_t)b * tiles + at.s0 / kScanTile) * a.channels + at.c0;
    for (int t = at.s0; t < at.end; t += kTT, buf ^= 1) {
        const int left = at.end - t;
        rB.store(sB[buf]);
        if constexpr (SEGS) rC.store(sC[buf]);
        float d[TPL], u[TPL], o[TPL];
        step_sizes<kTT, LPC, Tin>(dr, bias, a.softplus, left, at.j, d);
#pragma unroll
        for (int i = 0; i < TPL; ++i) u[i] = taken(d[i]) * widen<Tin>(xr[i]);
        float first = 0.f, second = 0.f;  // sums of the steps of the two tiles
        if constexpr (SEGS) {
#pragma unroll
            for (int i = 0; i < TPL; ++i) {
                const bool early = i * LPC + at.j < kScanTile;
                first += early ? d[i] : 0.f;
                second += early ? 0.f : d[i];
                o[i] = widen<Tdy>(gr[i]);
            }
            first = lane_total<LPC>(first);
            second = lane_total<LPC>(second);
            if (gate) {
#pragma unroll
                for (int i = 0; i < TPL; ++i) {
                    const float z = widen<Tin>(zr[i]);
                    o[i] *= z * logistic(z);
                }
            }
        }
        // the state before a tile
        auto keep = [&] {
            mine.store(tile_state + tile * NP, h);
            if (SEGS) mine.store_number(tile_steps + tile, steps);
            tile += a.channels;
        };
        __syncthreads();
        if (left > kTT) fetch(left - kTT);
        for_lanes<kTT>([&](auto T) {
            constexpr int tk = decltype(T)::value, i = tk / LPC, k = tk % LPC;
            if constexpr (tk == 0) {
                keep();
                steps += first;
            }
            if constexpr (tk == kScanTile) {
                keep();
                steps += second;
            }
            const float dk = lane_bcast<LPC, k>(d[i]), uk = lane_bcast<LPC, k>(u[i]);
            const floatx4 Bv = *reinterpret_cast<const floatx4 *>(&sB[buf][tk * NP + n0]);
            floatx4 Co;
            if constexpr (SEGS) {
                const float ok = lane_bcast<LPC, k>(o[i]);
                Co = *reinterpret_cast<const floatx4 *>(&sC[buf][tk * NP + n0]);
#pragma unroll
                for (int r = 0; r < 4; ++r) Co[r] *= ok;
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float e = fast_exp2(dk * A2[r]);
                h[r] = fmaf(e, h[r], uk * Bv[r]);
                if constexpr (SEGS) {
                    P[r] *= e;
                    Gs[r] = fmaf(P[r], Co[r], Gs[r]);
                }
            }
        });
    }
    if constexpr (SEGS) {
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
    const float A2 = ok ? rate(A[(int64_t)c * N + n]) : 0.f;
    const float *from = adj ? dfinal : init;
    const float h = carry_segments(ok && from != nullptr ? from[bcn] : 0.f, A2,
                                   (adj ? seg_adj : seg_state) + (int64_t)b * nseg * channels * NP + i,
                                   seg_steps + (int64_t)b * nseg * channels + c, (int64_t)channels * NP, channels, nseg,
                                   adj);
    if (adj && ok && dinit != nullptr) dinit[bcn] = h;
}

struct BwdOut {
    float *dx, *ddt, *dz, *dinit;
    float *db, *dc;         // dB and dC, or a block's partial rows of them
    int64_t blk, tok;       // elements between blocks and between tokens there
    float *dap, *ddp, *dbiasp;
    int runs;
};

// LDS row of one lane's 8 + 8 sums of a tile, padded by four words: the first
// words of 16 neighbouring rows lie on 16 different multiples of four modulo 64.
// So the 64 words that a wave reads of four columns differ modulo 64 at 16
// states; at 32 states two of them coincide, and at 64 four.  (Counted at 16
// states, 2 x 2048 tokens of 5120 channels: 1e7 conflict cycles over 7.5e6 LDS
// instructions of every kind, 16 us on each of 256 CUs.)
constexpr int kRedStride = 2 * kScanTile + 4;

// One segment, its tiles from the last to the first.  Registers limit it: a
// tile's states and decays take 8 a token, so tiles have 8 tokens (168
// registers at 16 states, two more spilled: three waves a SIMD; 16 tokens would
// leave one).
template <typename Tin, typename Tdy, int LPC>
__global__ __launch_bounds__(256, LPC == 4 ? 3 : 2)
void ks_bwd_main(ScanIn<Tin> a, const Tdy *__restrict__ dy, Strides dys,
                 const float *__restrict__ dfinal,
                 const float *__restrict__ seg_state,
                 const float *__restrict__ seg_adj,
                 const float *__restrict__ tile_state,
                 const float *__restrict__ tile_steps, int64_t tiles, BwdOut out) {
    constexpr int TT = kScanTile, NP = 4 * LPC, TPL = own_tokens<TT, LPC>();
    __shared__ float sB[TT * NP], sC[TT * NP], red[256 * kRedStride];
    const ScanPos<LPC> at(a);
    const int n0 = 4 * at.j, b = at.b, c = at.c;
    const int lane = threadIdx.x % 64;
    // LDS rows of sums: the parts of the waves, each of NP states
    const int red_row = threadIdx.x / 64 * 64 + channel_sum_part<LPC>(lane) * NP + n0 + channel_sum_r<LPC>(lane);
    const int64_t slot = ((int64_t)b * a.nseg + at.seg) * a.channels + c;
    const int64_t bc = (int64_t)b * a.channels + c;
    const bool segs = a.nseg > 1;
    float A2[4], carry[4], dA[4], hs[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        A2[r] = n0 + r < a.N ? rate(a.A[(int64_t)c * a.N + n0 + r]) : 0.f;
        dA[r] = hs[r] = 0.f;
    }
    if (segs) {
        load_states(seg_adj + slot * NP + n0, carry);
        load_states(seg_state + slot * NP + n0, hs);
    } else {
        load_states_n(dfinal != nullptr ? dfinal + bc * a.N : nullptr, n0, a.N, carry);
    }
    const float bias = a.bias != nullptr ? a.bias[c] : 0.f;
    const float D = a.D != nullptr ? a.D[c] : 0.f;
    const bool gate = a.z != nullptr;
    float dD = 0.f, dbias = 0.f;

    const int done = at.end > at.s0 ? at.s0 + (at.end - at.s0 + TT - 1) / TT * TT : at.s0;
    const int last = done - TT;
    // backwards through the tiles, offsets formed again at each (registers);
    // lanes without a channel read zeros: they add nothing to the sums over channels
    using InRows = OwnRows<TT, LPC, Tin, false, false>;
    using OutRows = OwnRows<TT, LPC, float, false, false>;
    InRows dts(a.dt, a.dts, b, c, at.j, at.ok, last), xs(a.x, a.xs, b, c, at.j, at.ok, last),
        zs(gate ? a.z : a.x, gate ? a.zs : a.xs, b, c, at.j, at.ok, last);
    OwnRows<TT, LPC, Tdy, false, false> gs(dy, dys, b, c, at.j, at.ok, last);
    const Strides dense{(int64_t)a.L * a.channels, a.channels};
    OutRows dxs(out.dx, dense, b, c, at.j, at.ok, last), ddts(out.ddt, dense, b, c, at.j, at.ok, last),
        dzs(gate ? out.dz : out.dx, dense, b, c, at.j, at.ok, last);
    RowStage<TT, NP, Tin, false> rB(a.B, a.Bs, b, at.g, a.N, last), rC(a.C, a.Cs, b, at.g, a.N, last);
    float *db = out.db + at.blk * out.blk, *dc = out.dc + at.blk * out.blk;

    // The sums over tokens leave a row for every kScanRun tokens of the segment, so that a sum in fp32 has no more
    // terms than that however time is cut, and start again.
    const BlockRows<LPC> mine(at.ok, at.j, at.cl);
    const int64_t run0 = ((int64_t)b * a.nseg + at.seg) * out.runs;
    auto leave_sums = [&](int run) {
        const int64_t row = (run0 + run) * a.channels + at.c0;
        mine.store(out.dap + row * NP, dA);
        mine.store_number(out.ddp + row, lane_total<LPC>(dD));
        mine.store_number(out.dbiasp + row, lane_total<LPC>(dbias));
#pragma unroll
        for (int r = 0; r < 4; ++r) dA[r] = 0.f;
        dD = dbias = 0.f;
    };
    for (int run = (done - at.s0 + kScanRun - 1) / kScanRun; run < out.runs; ++run) leave_sums(run);

    // rows behind the end
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

    uint32_t dr[TPL], xr[TPL], zr[TPL], gr[TPL];
    float hr[4], sr = 0.f;
    int64_t tile = ((int64_t)b * tiles + last / TT) * a.channels + at.c0;
    auto fetch = [&](int left) {
        dts.load(left, dr);
        xs.load(left, xr);
        if (gate) zs.load(left, zr);
        gs.load(left, gr);
        rB.load(left);
        rC.load(left);
        mine.load(tile_state + tile * NP, hr);
        if (segs) sr = mine.load_number(tile_steps + tile);
        tile -= a.channels;
        dts.next();
        xs.next();
        zs.next();
        gs.next();
        rB.next();
        rC.next();
    };
    if (at.s0 < at.end) fetch(at.end - last);
    for (int t = last; t >= at.s0; t -= TT) {
        const int left = at.end - t, room = at.s1 - t;
        rB.store(sB);
        rC.store(sC);
        float d[TPL], u[TPL], x[TPL], o[TPL], sl[TPL], zy[TPL], h0[4];
        step_sizes<TT, LPC, Tin>(dr, bias, a.softplus, left, at.j, d);
#pragma unroll
        for (int i = 0; i < TPL; ++i) {
            x[i] = widen<Tin>(xr[i]);
            u[i] = taken(d[i]) * x[i];
            o[i] = widen<Tdy>(gr[i]);
            sl[i] = a.softplus ? logistic(widen<Tin>(dr[i]) + bias) : 1.f;  // softplus'
        }
        if (gate) {
#pragma unroll
            for (int i = 0; i < TPL; ++i) {
                const float z = widen<Tin>(zr[i]), s = logistic(z);
                zy[i] = o[i] * (s * fmaf(z, 1.f - s, 1.f));  // dy silu'(z)
                o[i] *= z * s;
            }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) h0[r] = hr[r];
        if (segs) {
#pragma unroll
            for (int r = 0; r < 4; ++r) h0[r] = fmaf(fast_exp2(sr * A2[r]), hs[r], h0[r]);
        }
        __syncthreads();
        if (t - TT >= at.s0) fetch(TT);

        // B's and C's rows are read from LDS again on the way back: kept, they would take 64 registers
        auto Brow = [&](int tk) { return *reinterpret_cast<const floatx4 *>(&sB[tk * NP + n0]); };
        auto Crow = [&](int tk) { return *reinterpret_cast<const floatx4 *>(&sC[tk * NP + n0]); };
        float e[TT][4], h[TT][4], pY[TT], pA[TT], pB[TT], sums[2][TT], v[2][4];
        for_lanes<TT>([&](auto T) {
            constexpr int tk = decltype(T)::value, i = tk / LPC, k = tk % LPC;
            const float dk = lane_bcast<LPC, k>(d[i]), uk = lane_bcast<LPC, k>(u[i]), ok = lane_bcast<LPC, k>(o[i]);
            const floatx4 Bv = Brow(tk), Cv = Crow(tk);
            pY[tk] = 0.f;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                e[tk][r] = fast_exp2(dk * A2[r]);
                h[tk][r] = fmaf(e[tk][r], tk == 0 ? h0[r] : h[tk > 0 ? tk - 1 : 0][r], uk * Bv[r]);
                pY[tk] = fmaf(Cv[r], h[tk][r], pY[tk]);
                v[tk % 2][r] = ok * h[tk][r];
            }
            if constexpr (tk % 2 == 1) channel_sums<LPC>(v, sums[1][tk - 1], sums[1][tk]);
        });
        if (gate) {
#pragma unroll
            for (int i = 0; i < TPL; ++i) zy[i] *= fmaf(D, x[i], own_sum<TT, LPC>(pY, i, at.j));
            if (left < TT) {
#pragma unroll
                for (int i = 0; i < TPL; ++i) zy[i] = i * LPC + at.j < left ? zy[i] : 0.f;
            }
            dzs.store(room, zy);
        }
        // rows behind the end: the last state, should it not be finite, stays out of their products
        if (left < TT) {
#pragma unroll
            for (int tk = 0; tk < TT; ++tk)
#pragma unroll
                for (int r = 0; r < 4; ++r) h[tk][r] = tk + 1 < left ? h[tk][r] : 0.f;
        }
        asm volatile("" ::: "memory");
        for_lanes<TT>([&](auto K) {
            constexpr int tk = TT - 1 - decltype(K)::value, i = tk / LPC, k = tk % LPC;
            const float dk = lane_bcast<LPC, k>(d[i]), uk = lane_bcast<LPC, k>(u[i]), ok = lane_bcast<LPC, k>(o[i]);
            const floatx4 Bv = Brow(tk), Cv = Crow(tk);
            pB[tk] = pA[tk] = 0.f;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float G = fmaf(Cv[r], ok, carry[r]);
                v[tk % 2][r] = uk * G;
                pB[tk] = fmaf(G, Bv[r], pB[tk]);
                carry[r] = e[tk][r] * G;
                const float q = carry[r] * (tk == 0 ? h0[r] : h[tk > 0 ? tk - 1 : 0][r]);
                pA[tk] = fmaf(q, A2[r], pA[tk]);
                dA[r] = fmaf(q, dk, dA[r]);
            }
            if constexpr (tk % 2 == 0) channel_sums<LPC>(v, sums[0][tk], sums[0][tk + 1]);
        });

        float dxv[TPL], ddtv[TPL];
#pragma unroll
        for (int i = 0; i < TPL; ++i) {
            const float gB = own_sum<TT, LPC>(pB, i, at.j), gA = own_sum<TT, LPC>(pA, i, at.j);
            ddtv[i] = fmaf(0.6931471805599453f, gA, gB * x[i]) * sl[i];  // pA used log2(e) A
            dxv[i] = fmaf(gB, taken(d[i]), D * o[i]);
            dD = fmaf(o[i], x[i], dD);
        }
        // rows behind the end, where the states' part may be anything
        if (left < TT || TT < LPC) {
#pragma unroll
            for (int i = 0; i < TPL; ++i) {
                const bool live = i * LPC + at.j < min(left, TT);
                ddtv[i] = live ? ddtv[i] : 0.f;
                dxv[i] = live ? dxv[i] : 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < TPL; ++i) dbias += ddtv[i];
        dxs.store(room, dxv);
        ddts.store(room, ddtv);
        dxs.next();
        ddts.next();
        dzs.next();

#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int tk = 0; tk < TT; tk += 4)
                *reinterpret_cast<floatx4 *>(&red[red_row * kRedStride + q * TT + tk]) =
                    floatx4{sums[q][tk], sums[q][tk + 1], sums[q][tk + 2], sums[q][tk + 3]};
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * TT * NP; i += 256) {
            const int n = i % NP, column = i / NP, tok = column % TT;
            float s = 0.f;
#pragma unroll
            for (int q = 0; q < 256 / NP; ++q) s += red[(q * NP + n) * kRedStride + column];
            if (n < a.N && tok < room) {
                const int64_t p = ((int64_t)b * a.L + t + tok) * out.tok + n;
                (column < TT ? db : dc)[p] = tok < left ? s : 0.f;
            }
        }
        if ((t - at.s0) % kScanRun == 0) leave_sums((t - at.s0) / kScanRun);
    }

    if (a.nseg == 1 && out.dinit != nullptr && at.ok) store_states_n(out.dinit + bc * a.N, n0, a.N, carry);
}

// The last sums, in a fixed order and 64 bits: dA, dD and ddt_bias over batch,
// segments and runs; dB and dC over the blocks of each group (gblocks 1: written
// in place already).  Eight threads an output, each every eighth term, so that
// few outputs of many terms still have their loads in flight together.
struct BwdSums {
    const float *dap, *ddp, *dbiasp, *dbp, *dcp;
    float *dA, *dD, *ddt_bias, *dB, *dC;
    int64_t slots;        // batch * nseg * runs
    int64_t rows;         // batch * seqlen
    int channels, N, NP, ngroups, gblocks;
};
__global__ __launch_bounds__(256) void ks_bwd_sums(BwdSums s, ScanSums plan) {
    constexpr int COLS = kSumOutputs;
    __shared__ double part[256];
    const int slice = threadIdx.x / COLS;
    for (int64_t group = blockIdx.x; group < plan.groups; group += plan.blocks) {
        int64_t i = group * COLS + threadIdx.x % COLS;
        const float *from = nullptr;
        float *to = nullptr;
        int64_t terms = s.slots, stride = 0;
        if (i < plan.rates) {
            from = s.dap + i / s.N * s.NP + i % s.N;
            stride = (int64_t)s.channels * s.NP;
            to = s.dA + i;
        } else if ((i -= plan.rates) < 2 * (int64_t)s.channels) {
            const bool first = i < s.channels;
            const int64_t c = first ? i : i - s.channels;
            from = (first ? s.ddp : s.dbiasp) + c;
            stride = s.channels;
            to = first ? s.dD : s.ddt_bias;
            to = to != nullptr ? to + c : nullptr;
        } else if ((i -= 2 * (int64_t)s.channels) < 2 * plan.rows) {
            const bool first = i < plan.rows;
            if (!first) i -= plan.rows;
            const int64_t n = i % s.N, g = i / s.N % s.ngroups, row = i / ((int64_t)s.N * s.ngroups);
            from = (first ? s.dbp : s.dcp) + (g * s.gblocks * s.rows + row) * s.N + n;
            stride = s.rows * s.N;
            terms = s.gblocks;
            to = (first ? s.dB : s.dC) + i;
        }
        double v = 0.0;
        if (to != nullptr) {
#pragma unroll 8
            for (int64_t k = slice; k < terms; k += kSumSlices) v += (double)from[k * stride];
        }
        part[threadIdx.x] = v;
        __syncthreads();
        if (slice == 0 && to != nullptr) {
#pragma unroll
            for (int q = 1; q < kSumSlices; ++q) v += part[q * COLS + threadIdx.x];
            *to = (float)v;
        }
        __syncthreads();  // the next group's partial sums take this one's place
    }
}

template <typename Tin, typename Tdy, int LPC>
hipError_t bwd(const ScanArgs &a, const ScanPlan &plan, hipStream_t stream) {
    const ScanIn<Tin> in = scan_in<Tin>(a, plan);
    const Tdy *dy = static_cast<const Tdy *>(a.dy);
    const dim3 grid((unsigned)(plan.nblk * plan.nseg), (unsigned)a.batch);
    hipError_t e = hipSuccess;
    if (a.batch > 0) {
        const auto sweep = plan.nseg > 1 ? ks_bwd_sweep<Tin, Tdy, LPC, true> : ks_bwd_sweep<Tin, Tdy, LPC, false>;
        if (a.seqlen > 0) {
            e = launch_kernel(sweep, grid, dim3(256), 0, stream, LaunchEvents{}, in, dy, a.dys, a.init, a.seg_state,
                              a.seg_adj, a.seg_steps, a.tile_state, a.tile_steps, plan.tiles);
            if (e != hipSuccess) return e;
        }
        if (plan.nseg > 1) {
            const int64_t n = (int64_t)a.channels * plan.np;
            e = launch_kernel(ks_bwd_carry, dim3((unsigned)((n + 255) / 256), (unsigned)a.batch, 2), dim3(256), 0,
                              stream, LaunchEvents{}, a.A, a.init, a.dfinal, a.seg_state, a.seg_adj,
                              (const float *)a.seg_steps, a.dinit, a.channels, a.dstate, plan.np, plan.nseg);
            if (e != hipSuccess) return e;
        }
        BwdOut out{a.dx, a.ddt, a.dz, a.dinit, a.dbp, a.dcp, a.batch * a.seqlen * a.dstate, a.dstate,
                   a.dap, a.ddp, a.dbiasp, plan.runs};
        if (plan.gblocks == 1) {  // one block a group: its rows are the outputs'
            out.db = a.dB;
            out.dc = a.dC;
            out.blk = a.dstate;
            out.tok = (int64_t)a.ngroups * a.dstate;
        }
        e = launch_kernel(ks_bwd_main<Tin, Tdy, LPC>, grid, dim3(256), 0, stream, LaunchEvents{}, in, dy, a.dys,
                          a.dfinal, (const float *)a.seg_state, (const float *)a.seg_adj,
                          (const float *)a.tile_state, (const float *)a.tile_steps, plan.tiles, out);
        if (e != hipSuccess) return e;
    }
    const BwdSums s{a.dap, a.ddp, a.dbiasp, a.dbp, a.dcp, a.dA, a.dD, a.ddt_bias, a.dB, a.dC,
                    a.batch * plan.nseg * plan.runs, a.batch * a.seqlen, a.channels, a.dstate, plan.np, a.ngroups, plan.gblocks};
    const ScanSums sums = scan_sums(a.batch, a.seqlen, a.channels, a.dstate, a.ngroups, plan.gblocks);
    return launch_kernel(ks_bwd_sums, dim3(sums.blocks), dim3(256), 0, stream, LaunchEvents{}, s, sums);
}

template <typename Tin, typename Tdy>
hipError_t bwd_np(const ScanArgs &a, const ScanPlan &plan, hipStream_t s) {
    switch (plan.np) {
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
