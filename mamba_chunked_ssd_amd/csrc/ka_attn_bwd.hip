// ka_attn_bwd.hip -- gradients through sliding-window attention with sinks.
//
//   P_tj = exp(s_tj - lse_t) ,  dP_tj = dy_t . v_j ,  delta_t = dy_t . y_t ,
//   dS_tj = P_tj (dP_tj - delta_t) ,
//   dq_t = scale sum_j dS_tj k_j ,  dk_j = scale sum_t dS_tj q_t ,
//   dv_j = sum_t P_tj dy_t  (t of every head that shares j)
//
// Two kernels, each of which owns what it writes, so that no sum depends on an
// order of arrival: over the queries as the forward pass is laid out (dq, and
// delta on the way), and over the keys (dk, dv), which forms the scores again.
// A query that sees itself alone (token 0, or every one where window is 1 and
// there are no sinks) has no gradient through its scores: dP - delta is 0 there,
// which delta, a sum over the rounded y, would miss by its rounding.
//
// A key's block takes the queries that see it through the window.  Sinks are
// seen by every later query of the sequence too: those are cut into chunks, a
// block each, and their sums added by a third kernel.
//
// 2 x 2048 tokens, 40 heads of 64 over 8, a window of 512, 4 sinks, bf16: the call 124
// to 129 us (up to 382 TFLOP/s of 10 products of headdim a pair of tokens); under a
// kernel trace, which slows them, 54 us over the queries, 64 over the keys, 15 and 5
// for the sinks.  The 14 products that two kernels form could only be
// 10 with dq, or dk and dv, added up in memory.  Matrix instructions take 22 and 25 % of
// that time, vector ones 34 and 29 %: the rest is the waves' waiting, for LDS reads and
// for each other at the tiles' barriers (three or four tiles on their way instead of
// one: no faster, so not for copies).  Over the queries, a wave leaves out blocks of 32
// keys that none of its queries sees, not only whole tiles of 64: 59 to 55 us; tiles
// of 128 keys took 68.
#include <algorithm>

#include "ka_attn.h"

namespace ssd {
namespace {

constexpr int kQueries = 128;
// Blocks of 128 keys up to which blocks of 32 are taken, twice as many where the
// window covers the sequence.  One sequence, 16 heads over 8, 4 sinks, us of the
// backward pass by 128 and by 32:
//   bf16 heads of 32, window 512: 128 blocks 47, 42; 160 blocks 47, 48; all tokens: 256 blocks 156, 144; 320 blocks 181, 189
//     of 64:  128 blocks 59, 53; 160 blocks 60, 63; all tokens: 256 blocks 203, 196; 320 blocks 243, 266
//     of 128: 96 blocks 92, 80; 128 blocks 95, 93 (window 128: 62, 72); all tokens: 192 blocks 284, 240; 320 blocks 447, 511
//   fp32 heads of 32, window 128: 192 blocks 95, 85; 224 blocks 96, 99; all tokens: 384 blocks 1124, 1093
//     of 64:  160 blocks 162, 159; 224 blocks 165, 188; all tokens: 320 blocks 1779, 1661; 384 blocks 2155, 2247
//     of 128: 96 blocks 266, 209; 128 blocks 270, 256; 160 blocks 342, 364; all tokens: 192 blocks 2182, 2055; 256 blocks
//             2980, 3223
template <typename T, int D>
inline bool few_keys(int64_t blocks, int seqlen, int window) {
    constexpr int64_t most = sizeof(T) == 2 ? (D == 128 ? 96 : 128) : (D == 128 ? 112 : 192);
    return blocks <= (window >= seqlen ? 2 * most : most);
}

template <typename T>
struct AttnBwdIn {
    const T *q, *k, *v, *y, *dy;
    const float *lse;
    const int32_t *lengths;
    T *dq, *dk, *dv;
    float2 *stats;  // (batch, heads, seqlen): lse in units of log(2), delta
    float *partials;
    HeadStrides qs, ks, vs, ys, dys;
    int L, heads, kvheads;
    int window, sinks;
    int sink_tiles, chunk, nchunks;  // of kSinkKeys keys; queries
    int64_t rows;  // of partial sums
    float scale, c;
};

__device__ __forceinline__ int length_of(const int32_t *lengths, int b, int L) {
    return lengths == nullptr ? L : min(max(lengths[b], 0), L);
}

// Elements 32 db .. of a wave's dq formed again (see with_odd): queries w0 .. w0
// + 31 below `len`, a lane's t.  Under a finite lse a key that is not finite has a
// weight and a dS of 0, which make NaN of it.
template <typename T, int D>
__device__ __forceinline__ void query_again(const AttnBwdIn<T> &a, const T *kh, const T *vh, const Frag<T> (&q)[D / 16],
                                            const Frag<T> (&dy)[D / 16], int w0, int len, int t, int db, float lse, float delta,
                                            T *row, bool on) {
    const int lane = threadIdx.x & 63, col = lane & 31, h = lane >> 5;
    const int near = max(w0 - a.window + 1, 0), last = min(w0 + 31, len - 1), far = min(a.sinks, near);
    const int nfar = (far + 31) / 32, blocks = nfar + (last - near) / 32 + 1;
    const bool alone = t == 0 || (a.window == 1 && a.sinks == 0);
    floatx16 o = zero16();
    uint32_t odd = 0;
#pragma unroll 1
    for (int n = 0; n < blocks; ++n) {
        const int j0 = n < nfar ? 32 * n : near + 32 * (n - nfar), stop = n < nfar ? far : last + 1;
        floatx16 s = zero16(), g = zero16();
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            Frag<T> f;
            load_frag(f, kh + (int64_t)(j0 + col) * a.ks.row + 16 * ks + 8 * h, j0 + col < stop);
            s = mma(f, q[ks], s);
            load_frag(f, vh + (int64_t)(j0 + col) * a.vs.row + 16 * ks + 8 * h, j0 + col < stop);
            g = mma(f, dy[ks], g);
        }
        const int upto = min(t, stop - 1) - j0 - 4 * h, before = t - a.window - j0 - 4 * h, sunk = a.sinks - j0 - 4 * h;
        Frag<T> sf[2], uf[2];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            float ds[8], u[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = 8 * ks + i, at = place(0, r);
                const bool seen = (at <= upto) & ((at > before) | (at < sunk));
                ds[i] = (seen & !alone) ? fast_exp2(fmaf(s[r], a.c, -lse)) * (g[r] - delta) : 0.f;
                u[i] = seen ? kOddNan : 0.f;
            }
            to_frag(ds, sf[ks]);
            to_frag(u, uf[ks]);
        }
        group_end();
        floatx16 kinds = zero16();
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            Frag<T> kf, kind;
            load_apart(kf, kind, 32 * db + col, [&](int i) {
                const int j = j0 + 16 * ks + 4 * h + i;
                return j < stop ? kh + (int64_t)j * a.ks.row : nullptr;
            });
            o = mma(kf, sf[ks], o);
            kinds = mma(kind, uf[ks], kinds);
            group_end();
        }
        odd |= odd_of(kinds);
    }
    float v[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) v[r] = with_odd(o[r] * a.scale, odd, r);
    store_column(row, db, h, v, on);
}

// SHARED (few queries): the waves of a block share 32 queries and take the
// tiles in turn, with stages of their own; their sums are added at the end, in
// order.  Else each has 32, and all use the same tiles.
// (bf16 heads of 32 are held to four waves a SIMD: at five, what forms rows again
// spills into the loop, 86 us the backward pass of 4 x 2048 tokens for 83.)
template <typename T, int D, bool SHARED>
__global__ __launch_bounds__((SHARED ? 64 * WaveLds<T, D>::kWaves : 256), (SHARED || D * sizeof(T) > 256 ? 1 : D * sizeof(T) > 64 ? 2 : 4)) void attn_dq_kernel(
    const AttnBwdIn<T> a) {
    constexpr int KT = sizeof(T) == 2 && !SHARED ? 64 : 32, KB = KT / 32, NS = D / 16, DB = D / 32;
    constexpr int NW = SHARED ? WaveLds<T, D>::kWaves : 4, kRun = SHARED ? 32 : kQueries;
    typedef Tile<T, D, KT> Tl;
    extern __shared__ __align__(16) unsigned char lds[];  // (the stages; SHARED: which queries to form again)

    const int group = a.heads / a.kvheads;
    const int tiles = (a.L + kRun - 1) / kRun;
    int n = xcd_remap((int)blockIdx.x, (int)gridDim.x);
    const int gh = n % group;
    n /= group;
    const int q0 = (tiles - 1 - n % tiles) * kRun;
    n /= tiles;
    const int kvh = n % a.kvheads, b = n / a.kvheads, head = kvh * group + gh;
    const int len = length_of(a.lengths, b, a.L);
    const int lane = threadIdx.x & 63, col = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int w0 = SHARED ? q0 : q0 + 32 * wave, t = w0 + col;  // the wave's queries
    const bool live = t < len;
    const int64_t dense = ((int64_t)b * a.L + t) * a.heads * D + (int64_t)head * D;
    const int64_t stat = ((int64_t)b * a.heads + head) * a.L + t;
    if (q0 >= len) {
        if (SHARED && wave > 0) return;
        const float z[16] = {};
        for (int db = 0; db < DB; ++db) store_column(a.dq + dense, db, h, z, t < a.L);
        return;
    }

    Frag<T> qf[NS], df[NS];
    float delta = 0.f;
    const T *qrow = a.q + (int64_t)b * a.qs.batch + (int64_t)t * a.qs.row + head * a.qs.head;
    const T *drow = a.dy + (int64_t)b * a.dys.batch + (int64_t)t * a.dys.row + head * a.dys.head;
    const T *yrow = a.y + (int64_t)b * a.ys.batch + (int64_t)t * a.ys.row + head * a.ys.head;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
        load_frag(qf[s], qrow + 16 * s + 8 * h, live);
        load_frag(df[s], drow + 16 * s + 8 * h, live);
    }
#pragma unroll
    for (int s = 0; s < NS; ++s) {
        Frag<T> yf;
        load_frag(yf, yrow + 16 * s + 8 * h, live);
        delta = dot_frag(df[s], yf, delta);
    }
    delta = both_halves(delta);
    const float lse = live ? a.lse[stat] * kLog2e : 0.f;
    if (live && h == 0 && (!SHARED || wave == 0)) a.stats[stat] = float2{lse, delta};

    const Walk<KT> walk(q0, min(q0 + kRun, len) - 1, 0, a.window, a.sinks);
    const T *kh = a.k + (int64_t)b * a.ks.batch + kvh * a.ks.head, *vh = a.v + (int64_t)b * a.vs.batch + kvh * a.vs.head;
    Copier<Tl, SHARED ? 1 : 4> kcopy, vcopy;
    kcopy.init(a.ks.row * (int64_t)sizeof(T), SHARED ? 0 : wave, lane);
    vcopy.init(a.vs.row * (int64_t)sizeof(T), SHARED ? 0 : wave, lane);
    unsigned char *own = lds + (SHARED ? wave * 4 * Tl::kBytes : 0);  // (2 stages, keys and values)
    const auto stage = [&](int n, int buf) {
        const int j0 = walk.start(n), rows = min((n < walk.nsink ? walk.sunk : len) - j0, KT);
        const uint32_t kl = lds_addr(own + buf * 2 * Tl::kBytes);
        kcopy.copy(kl, kh + (int64_t)j0 * a.ks.row, rows);
        vcopy.copy(kl + Tl::kBytes, vh + (int64_t)j0 * a.vs.row, rows);
    };
    constexpr int kStep = SHARED ? NW : 1;
    const int first = SHARED ? wave : 0;
    if (first < walk.ntiles) stage(first, 0);

#pragma unroll
    for (int s = 0; s < NS; ++s) {
        arrived(qf[s]);
        arrived(df[s]);
    }
    floatx16 o[DB];
#pragma unroll
    for (int db = 0; db < DB; ++db) o[db] = zero16();
    const int w1 = min(w0 + 31, len - 1);
    const bool alone = t == 0 || (a.window == 1 && a.sinks == 0);  // (such a row's tile is never whole)
    int buf = 0;
    for (int n = first; n < walk.ntiles; n += kStep, buf ^= 1) {
        // (what was read of the other stage has arrived too)
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        if constexpr (!SHARED) __syncthreads();
        if (n + kStep < walk.ntiles) stage(n + kStep, buf ^ 1);
        if (w0 >= len) continue;
        const unsigned char *kl = own + buf * 2 * Tl::kBytes, *vl = kl + Tl::kBytes;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            const int j0 = walk.start(n) + 32 * kb;
            if (j0 > w1 || (n < walk.nsink ? j0 >= walk.sunk : j0 + 32 <= w0 - a.window + 1 && j0 >= a.sinks)) continue;
            const bool whole = n < walk.nsink ? j0 + 32 <= walk.sunk
                                              : j0 + 31 <= w0 && (w0 + 31 - j0 < a.window || j0 + 32 <= a.sinks);
            floatx16 s, g;
            both_scores<Tl>(kl + Tl::at(32 * kb, 0), vl + Tl::at(32 * kb, 0), qf, df, lane, s, g);
            Frag<T> kf[2][DB];
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                for (int db = 0; db < DB; ++db) Tl::across(kl, 32 * kb + 16 * ks, 32 * db, lane, kf[ks][db]);
            group_end();
            float ds[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) ds[r] = fast_exp2(fmaf(s[r], a.c, -lse)) * (g[r] - delta);
            if (!whole) {
                // (a tile of sinks: all of them, up to its end)
                const Mask mask(n < walk.nsink ? walk.sunk - 1 : t, j0, h, n < walk.nsink ? kAttnFar : a.window, a.sinks);
#pragma unroll
                for (int r = 0; r < 16; ++r) ds[r] = (mask.seen(place(0, r)) & !alone) ? ds[r] : 0.f;
            }
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                Frag<T> sf;
                to_frag(reinterpret_cast<const float(&)[8]>(ds[8 * ks]), sf);
#pragma unroll
                for (int db = 0; db < DB; ++db) o[db] = mma(kf[ks][db], sf, o[db]);
            }
        }
    }
    if constexpr (SHARED) {
        floatx4 *sums = reinterpret_cast<floatx4 *>(lds) + lane;  // (wave, register quad, lane)
        __syncthreads();
        if (wave > 0) {
#pragma unroll
            for (int q = 0; q < DB * 4; ++q)
                sums[((wave - 1) * DB * 4 + q) * 64] = floatx4{o[q / 4][4 * (q % 4)], o[q / 4][4 * (q % 4) + 1], o[q / 4][4 * (q % 4) + 2], o[q / 4][4 * (q % 4) + 3]};
        }
        __syncthreads();
        if (wave == 0) {
#pragma unroll
            for (int of = 0; of < NW - 1; ++of)
#pragma unroll
                for (int q = 0; q < DB * 4; ++q) {
                    const floatx4 x = sums[(of * DB * 4 + q) * 64];
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[q / 4][4 * (q % 4) + e] += x[e];
                }
        }
    }
    if (w0 >= a.L) return;  // (not SHARED: no barrier follows)

    float check = 0.f;
    if (!SHARED || wave == 0) {
#pragma unroll
        for (int db = 0; db < DB; ++db) {
            float v[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                check = fmaf(o[db][r], 0.f, check);
                v[r] = live ? o[db][r] * a.scale : 0.f;
            }
            store_column(a.dq + dense, db, h, v, t < a.L);
        }
    }
    // As in the forward pass: rows that a value they do not see may have spoiled.
    check = both_halves(check);
    uint32_t again = (uint32_t)__ballot(live && check != check && delta - delta == 0.f && lse - lse == 0.f);
    if constexpr (SHARED) {
        // by all waves, which take some of the elements each
        uint32_t *told = reinterpret_cast<uint32_t *>(lds + WaveLds<T, D>::kCopies);
        if (threadIdx.x == 0) *told = again;
        __syncthreads();
        again = *told;
    }
    if (again != 0) {
#pragma unroll 1
        for (int db = SHARED ? wave : 0; db < DB; db += SHARED ? NW : 1)
            query_again<T, D>(a, kh, vh, qf, df, w0, len, t, db, lse, delta, a.dq + dense, (again >> col & 1) != 0);
    }
}

// KW waves of 32 keys each, which they hold in registers (columns of the
// products S = Q K^T, dP = dY V^T), G times over: against tiles of 32 G QB
// queries, of which each group of waves takes its own blocks of 32, one tile on
// the way while another is in use.  dv^T += dY^T P and dk^T += Q^T dS take the
// same tiles across.  The groups' sums are added at the end, in order.
//
// A block's queries are all those that see its keys through the window, or a
// chunk of those that see them as sinks alone (blocks behind `tiles`).
enum class Part { window, sinks, both };

// Elements 32 db .. of a wave's dk and dv formed again (see with_odd): a lane's
// key j of w0 .. w0 + 31, over the queries lo .. hi - 1 of the group's heads that
// see it through the window (far: as a sink alone).  A query that is not finite
// makes NaN of every weight in its row; where its own key is all that it sees, dS
// is 0 and 0 times it is NaN.
template <typename T, int D>
__device__ __forceinline__ void keys_again(const AttnBwdIn<T> &a, const T *q, const T *dy, const float2 *stats, int group,
                                           const Frag<T> (&k)[D / 16], const Frag<T> (&v)[D / 16], int w0, int j, int lo, int hi,
                                           bool far, int db, floatx16 &dk, floatx16 &dv) {
    const int lane = threadIdx.x & 63, col = lane & 31, h = lane >> 5;
    const bool lone = a.window == 1 && a.sinks == 0;
    // of the wave's keys; a lane's own
    const int from = max(lo, far ? w0 + a.window : w0);
    const int to = far ? (w0 < a.sinks ? hi : from) : (int)min((int64_t)hi, (int64_t)w0 + 31 + a.window);
    const int first = far ? j + a.window : j;
    const int last = far ? (j < a.sinks ? to : first) - 1 : (int)min((int64_t)to, (int64_t)j + a.window) - 1;
    uint32_t kodd = 0, vodd = 0;
    dk = dv = zero16();
    for (int head = 0; head < group; ++head, q += a.qs.head, dy += a.dys.head, stats += a.L) {
#pragma unroll 1
        for (int t0 = from; t0 < to; t0 += 32) {
            floatx16 s = zero16(), g = zero16(), kinds = zero16(), vinds = zero16();
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                Frag<T> f;
                load_frag(f, q + (int64_t)(t0 + col) * a.qs.row + 16 * ks + 8 * h, t0 + col < to);
                s = mma(f, k[ks], s);
                load_frag(f, dy + (int64_t)(t0 + col) * a.dys.row + 16 * ks + 8 * h, t0 + col < to);
                g = mma(f, v[ks], g);
            }
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                float p[8], ds[8], pu[8], su[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int r = 8 * ks + i, t = t0 + 4 * h + place(0, r);
                    const bool seen = (t >= first) & (t <= last);
                    const float2 st = seen ? stats[t] : float2{0.f, 0.f};
                    p[i] = seen ? fast_exp2(fmaf(s[r], a.c, -st.x)) : 0.f;
                    ds[i] = (seen & (t > 0) & !lone) ? p[i] * (g[r] - st.y) : 0.f;
                    pu[i] = !seen ? 0.f : s[r] == -kInf ? kOddNan : 1.f;
                    su[i] = seen ? kOddNan : 0.f;
                }
                const auto add = [&](const T *x, int64_t stride, const float (&weight)[8], const float (&one)[8], floatx16 &sum,
                                     floatx16 &kinds, uint32_t &odd) {
                    Frag<T> w, u, f, kind;
                    to_frag(weight, w);
                    to_frag(one, u);
                    load_apart(f, kind, 32 * db + col, [&](int i) {
                        const int t = t0 + 16 * ks + 4 * h + i;
                        return t < to ? x + (int64_t)t * stride : nullptr;
                    });
                    sum = mma(f, w, sum);
                    // (fp32 heads of 128 have no registers to hold kinds in)
                    if constexpr (D * sizeof(T) > 256) odd |= odd_of(mma(kind, u, zero16()));
                    else kinds = mma(kind, u, kinds);
                    group_end();
                };
                add(dy, a.dys.row, p, pu, dv, vinds, vodd);
                add(q, a.qs.row, ds, su, dk, kinds, kodd);
            }
            if constexpr (D * sizeof(T) <= 256) {
                kodd |= odd_of(kinds);
                vodd |= odd_of(vinds);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        dk[r] = with_odd(dk[r] * a.scale, kodd, r);
        dv[r] = with_odd(dv[r], vodd, r);
    }
}

template <typename T, int D, int KW, int G, int QB>
struct KeyLds {
    typedef Tile<T, D, 32 * G * QB> Tl;
    static constexpr int kStats = Tl::kBytes * 2, kStage = kStats + 32 * G * QB * (int)sizeof(float2);
    static constexpr int kSums = G > 1 ? KW * D * 256 : 0;  // of one group
    static constexpr int kTold = 2 * kStage > kSums ? 2 * kStage : kSums;  // which keys to form again, a word for each KW
    static constexpr int kBytes = kTold + 16;
};

template <typename T, int D, int KW, int G, int QB, Part PART>
__global__ __launch_bounds__((64 * KW * G), 1) void attn_dkv_kernel(const AttnBwdIn<T> a) {
    constexpr int NS = D / 16, DB = D / 32, NW = KW * G, QT = 32 * G * QB;
    typedef KeyLds<T, D, KW, G, QB> Lds;
    typedef typename Lds::Tl Tl;
    extern __shared__ __align__(16) unsigned char lds[];  // (2 stages: queries, dy, stats); then a group's sums

    const int group = a.heads / a.kvheads, tiles = PART == Part::sinks ? 0 : (a.L + 32 * KW - 1) / (32 * KW);
    const int items = tiles + (PART == Part::window ? 0 : a.sink_tiles * a.nchunks);
    int n = xcd_remap((int)blockIdx.x, (int)gridDim.x);
    const int item = n % items;
    n /= items;
    const int kvh = n % a.kvheads, b = n / a.kvheads;
    const int len = length_of(a.lengths, b, a.L);
    const bool far = PART == Part::both ? item >= tiles : PART == Part::sinks;
    const int part = far ? 1 + (item - tiles) % a.nchunks : 0, j0 = (far ? (item - tiles) / a.nchunks : item) * 32 * KW;
    const int lo = far ? max(a.window + (part - 1) * a.chunk, a.window + j0) : j0;
    const int hi = far ? min(len, a.window + part * a.chunk) : (int)min((int64_t)len, (int64_t)j0 + 32 * KW - 1 + a.window);
    const int turns = hi > lo ? (hi - lo + QT - 1) / QT * group : 0;

    const int lane = threadIdx.x & 63, col = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), part_of = wave / KW;  // which group
    const int w0 = j0 + 32 * (wave % KW), j = w0 + col;
    const bool live = j < len;
    const T *kh = a.k + (int64_t)b * a.ks.batch + kvh * a.ks.head, *vh = a.v + (int64_t)b * a.vs.batch + kvh * a.vs.head;
    const T *qb = a.q + (int64_t)b * a.qs.batch, *db_ = a.dy + (int64_t)b * a.dys.batch;
    Frag<T> kf[NS], vf[NS];
#pragma unroll
    for (int s = 0; s < NS; ++s) {
        load_frag(kf[s], kh + (int64_t)j * a.ks.row + 16 * s + 8 * h, live);
        load_frag(vf[s], vh + (int64_t)j * a.vs.row + 16 * s + 8 * h, live);
    }

    Copier<Tl, NW> qcopy, dcopy;
    qcopy.init(a.qs.row * (int64_t)sizeof(T), wave, lane);
    dcopy.init(a.dys.row * (int64_t)sizeof(T), wave, lane);
    int head = kvh * group, next = lo;  // of the tile to stage
    const auto stage = [&](int buf) {
        const int rows = min(hi - next, QT);
        const uint32_t to = lds_addr(lds + buf * Lds::kStage);
        qcopy.copy(to, qb + (int64_t)next * a.qs.row + head * a.qs.head, rows);
        dcopy.copy(to + Tl::kBytes, db_ + (int64_t)next * a.dys.row + head * a.dys.head, rows);
        if (wave < QT / 32) {
            const i32x4 desc = buffer_desc(a.stats + ((int64_t)b * a.heads + head) * a.L + next, (uint32_t)rows * (uint32_t)sizeof(float2));
            lds_dma_x1(desc, to + Lds::kStats + 256 * wave, 256 * wave + 4 * lane);
        }
        next += QT;
        if (next >= hi) {
            next = lo;
            ++head;
        }
    };
    if (turns > 0) stage(0);

#pragma unroll
    for (int s = 0; s < NS; ++s) {
        arrived(kf[s]);
        arrived(vf[s]);
    }
    const bool lone = a.window == 1 && a.sinks == 0;
    floatx16 dk[DB], dv[DB];
#pragma unroll
    for (int db = 0; db < DB; ++db) dk[db] = dv[db] = zero16();
    int tile = lo;
    for (int n = 0; n < turns; ++n) {
        lds_dma_wait();
        __syncthreads();
        if (n + 1 < turns) stage((n + 1) & 1);
        const unsigned char *ql = lds + (n & 1) * Lds::kStage, *dl = ql + Tl::kBytes;
        const float2 *stats = reinterpret_cast<const float2 *>(ql + Lds::kStats);
#pragma unroll
        for (int qi = 0; qi < QB; ++qi) {
            const int q0 = 32 * (part_of * QB + qi), t0 = tile + q0;
            if (far ? w0 >= a.sinks || t0 + 31 - w0 < a.window : t0 + 31 < w0 || t0 - w0 - 31 >= a.window) continue;
            if (t0 >= hi) continue;
            const bool whole = far ? w0 + 32 <= a.sinks && t0 - w0 - 31 >= a.window : t0 >= w0 + 31 && t0 + 31 - w0 < a.window;
            floatx16 s, g;
            both_scores<Tl>(ql + Tl::at(q0, 0), dl + Tl::at(q0, 0), kf, vf, lane, s, g);
            floatx4 st[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) st[r] = *reinterpret_cast<const floatx4 *>(stats + q0 + place(0, 2 * r) + 4 * h);
            Frag<T> f[2][DB];
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                for (int db = 0; db < DB; ++db) Tl::across(dl, q0 + 16 * ks, 32 * db, lane, f[ks][db]);
            group_end();
            float p[16], ds[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                p[r] = fast_exp2(fmaf(s[r], a.c, -st[r / 2][2 * (r % 2)]));
                ds[r] = p[r] * (g[r] - st[r / 2][2 * (r % 2) + 1]);
            }
            if (!whole) {
                // rows are queries here: t - j within a window of the key's
                const int back = t0 + 4 * h - j, left = hi - t0 - 4 * h, sunk = j < a.sinks ? 0 : kAttnFar;
                const int first = t0 == 0 ? -4 * h : -1;
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int at = place(0, r), d = at + back;
                    const bool on = far ? (at < left) & (d >= a.window + sunk) : (at < left) & (d >= 0) & (d < a.window);
                    p[r] = on ? p[r] : 0.f;
                    ds[r] = (on & (at != first) & !lone) ? ds[r] : 0.f;
                }
            }
            Frag<T> f2[2][DB];
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                Frag<T> pf;
                to_frag(reinterpret_cast<const float(&)[8]>(p[8 * ks]), pf);
#pragma unroll
                for (int db = 0; db < DB; ++db) {
                    Tl::across(ql, q0 + 16 * ks, 32 * db, lane, f2[ks][db]);
                    dv[db] = mma(f[ks][db], pf, dv[db]);
                }
            }
            group_end();
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                Frag<T> sf;
                to_frag(reinterpret_cast<const float(&)[8]>(ds[8 * ks]), sf);
#pragma unroll
                for (int db = 0; db < DB; ++db) dk[db] = mma(f2[ks][db], sf, dk[db]);
            }
        }
        tile += QT;
        if (tile >= hi) tile = lo;
    }
#pragma unroll
    for (int of = 1; of < G; ++of) {
        floatx4 *sums = reinterpret_cast<floatx4 *>(lds) + (wave % KW) * D * 16 + lane;  // (register quad, lane)
        __syncthreads();
        if (part_of == of) {
#pragma unroll
            for (int db = 0; db < DB; ++db)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sums[(db * 8 + i) * 64] = floatx4{dk[db][4 * i], dk[db][4 * i + 1], dk[db][4 * i + 2], dk[db][4 * i + 3]};
                    sums[(db * 8 + 4 + i) * 64] = floatx4{dv[db][4 * i], dv[db][4 * i + 1], dv[db][4 * i + 2], dv[db][4 * i + 3]};
                }
        }
        __syncthreads();
        if (part_of == 0) {
#pragma unroll
            for (int db = 0; db < DB; ++db)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const floatx4 x = sums[(db * 8 + i) * 64], y = sums[(db * 8 + 4 + i) * 64];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        dk[db][4 * i + e] += x[e];
                        dv[db][4 * i + e] += y[e];
                    }
                }
        }
    }

    const bool partial = far || w0 < a.rows;
    const int64_t dense = ((int64_t)b * a.L + j) * a.kvheads * D + (int64_t)kvh * D;
    float *pk = a.partials + ((((int64_t)b * a.kvheads + kvh) * (1 + a.nchunks) + part) * 2 * a.rows + j) * D;
    float *pv = pk + a.rows * D;
    const auto write = [&](int db, const floatx16 &dk, const floatx16 &dv, float k_scale, bool on) {
        float x[16], z[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            x[r] = live ? dk[r] * k_scale : 0.f;
            z[r] = live ? dv[r] : 0.f;
        }
        if (partial) {
            store_column(pk, db, h, x, on);
            store_column(pv, db, h, z, on);
        } else {
            store_column(a.dk + dense, db, h, x, on && j < a.L);
            store_column(a.dv + dense, db, h, z, on && j < a.L);
        }
    };
    float check = 0.f;
    if (part_of == 0 && w0 < a.L) {
#pragma unroll
        for (int db = 0; db < DB; ++db) {
#pragma unroll
            for (int r = 0; r < 16; ++r) check = fmaf(dk[db][r], 0.f, fmaf(dv[db][r], 0.f, check));
            write(db, dk[db], dv[db], a.scale, true);
        }
    }
    // Keys that a query which does not see them may have spoiled, by all groups, which take some of the elements each.
    check = both_halves(check);
    uint32_t again = (uint32_t)__ballot(live && check != check);
    if constexpr (G > 1) {
        uint32_t *told = reinterpret_cast<uint32_t *>(lds + Lds::kTold) + wave % KW;
        if (part_of == 0 && lane == 0) *told = again;
        __syncthreads();
        again = *told;
    }
    if (again != 0) {
#pragma unroll 1
        for (int db = part_of; db < DB; db += G) {
            floatx16 x, z;
            keys_again<T, D>(a, qb + kvh * group * a.qs.head, db_ + kvh * group * a.dys.head,
                             a.stats + ((int64_t)b * a.heads + kvh * group) * a.L, group, kf, vf, w0, j, lo, hi, far, db, x, z);
            write(db, x, z, 1.f, (again >> col & 1) != 0);
        }
    }
}

// The sink tiles' rows of dk and dv: the window's part and the chunks', in that order.
template <typename T>
__global__ __launch_bounds__(256) void attn_sinks_kernel(const AttnBwdIn<T> a, int64_t heads, int D) {
    const int64_t keys = min((int64_t)a.L, a.rows), parts = 1 + a.nchunks, all = 2 * heads * keys * D;
    for (int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x; n < all; n += (int64_t)gridDim.x * 256) {
        const int e = (int)(n % D);
        int64_t rest = n / D;
        const int64_t j = rest % keys;
        rest /= keys;
        const int64_t of = rest >> 1, b = of / a.kvheads, kvh = of % a.kvheads;  // head of keys among all sequences'
        const bool second = (rest & 1) != 0;
        const float *p = a.partials + ((of * parts * 2 + second) * a.rows + j) * D + e;
        float s = 0.f;
#pragma unroll 8
        for (int k = 0; k < parts; ++k) s += p[k * 2 * a.rows * D];
        narrow((second ? a.dv : a.dk) + ((b * a.L + j) * a.kvheads + kvh) * D + e, s);
    }
}

template <typename T, int D, int KW, int G, int QB, Part PART>
hipError_t attn_dkv_launch(const AttnBwdIn<T> &in, int64_t blocks, hipStream_t stream) {
    constexpr int kLds = KeyLds<T, D, KW, G, QB>::kBytes;
    const hipError_t e = allow_lds<attn_dkv_kernel<T, D, KW, G, QB, PART>>(kLds);
    if (e != hipSuccess) return e;
    attn_dkv_kernel<T, D, KW, G, QB, PART><<<dim3((uint32_t)blocks), dim3(64 * KW * G), kLds, stream>>>(in);
    return hipGetLastError();
}

template <typename T, int D>
hipError_t attn_bwd_sized(const AttnBwdIn<T> &in, int64_t batch, hipStream_t stream) {
    constexpr int kLds = 2 * 2 * Tile<T, D, sizeof(T) == 2 ? 64 : 32>::kBytes;
    // two groups of waves where a wave's registers (keys, values, their gradients) leave room for two on a SIMD
    constexpr bool kSmall = D * sizeof(T) <= 128;
    // blocks of queries for a wave and tile, bf16 heads of 64: one 75 us, two 64, four 67
    constexpr int G = kSmall ? 2 : 1, QB = sizeof(T) == 2 ? 2 : 1, GS = D * sizeof(T) <= 256 ? 4 : 2;
    // fewer blocks of 128 than compute units: blocks of 32, whose waves share them and part the rest
    const int64_t rows = batch * in.heads, qblocks = rows * ((in.L + kQueries - 1) / kQueries);
    hipError_t e;
    if (few_queries<T, D>(qblocks, in.L, in.window, false)) {
        constexpr int kWaveLds = WaveLds<T, D>::kCopies + 16;
        e = allow_lds<attn_dq_kernel<T, D, true>>(kWaveLds);
        if (e != hipSuccess) return e;
        attn_dq_kernel<T, D, true><<<dim3((uint32_t)(rows * ((in.L + 31) / 32))), dim3(64 * WaveLds<T, D>::kWaves), kWaveLds, stream>>>(in);
    } else {
        e = allow_lds<attn_dq_kernel<T, D, false>>(kLds);
        if (e != hipSuccess) return e;
        attn_dq_kernel<T, D, false><<<dim3((uint32_t)qblocks), dim3(256), kLds, stream>>>(in);
    }
    if ((e = hipGetLastError()) != hipSuccess) return e;
    const int64_t heads = batch * in.kvheads;
    const int64_t blocks = heads * ((in.L + 127) / 128);
    const int64_t chunks = heads * in.sink_tiles * in.nchunks;
    if (few_keys<T, D>(blocks, in.L, in.window)) {
        // blocks of 32 keys, whose waves share them and part the queries; the sinks' among them
        e = attn_dkv_launch<T, D, 1, GS, 1, Part::both>(in, heads * ((in.L + 31) / 32) + chunks, stream);
    } else {
        e = attn_dkv_launch<T, D, 4, G, QB, Part::window>(in, blocks, stream);
        if (e == hipSuccess && chunks > 0) e = attn_dkv_launch<T, D, 1, GS, 1, Part::sinks>(in, chunks, stream);
    }
    if (e != hipSuccess || chunks == 0) return e;
    const int64_t n = 2 * heads * std::min<int64_t>(in.L, in.rows) * D;
    attn_sinks_kernel<T><<<dim3((uint32_t)std::min<int64_t>((n + 255) / 256, 1 << 16)), dim3(256), 0, stream>>>(in, heads, D);
    return hipGetLastError();
}

template <typename T>
hipError_t attn_bwd_typed(const AttnArgs &a, const AttnBwdPlan &p, hipStream_t stream) {
    const AttnBwdIn<T> in{static_cast<const T *>(a.q), static_cast<const T *>(a.k), static_cast<const T *>(a.v),
                          static_cast<const T *>(a.y), static_cast<const T *>(a.dy), a.lse, a.lengths,
                          static_cast<T *>(a.dq), static_cast<T *>(a.dk), static_cast<T *>(a.dv), reinterpret_cast<float2 *>(a.stats), a.partials,
                          a.qs, a.ks, a.vs, a.ys, a.dys, a.seqlen, a.heads, a.kvheads,
                          a.window, a.sinks, p.sink_tiles, p.chunk, p.nchunks, p.rows, a.scale, a.scale * kLog2e};
    return a.headdim == 32   ? attn_bwd_sized<T, 32>(in, a.batch, stream)
           : a.headdim == 64 ? attn_bwd_sized<T, 64>(in, a.batch, stream)
                             : attn_bwd_sized<T, 128>(in, a.batch, stream);
}

}  // namespace

hipError_t launch_attn_bwd(const AttnArgs &a, const AttnBwdPlan &plan, hipStream_t stream) {
    return a.bf16 ? attn_bwd_typed<uint16_t>(a, plan, stream) : attn_bwd_typed<float>(a, plan, stream);
}

}  // namespace ssd
