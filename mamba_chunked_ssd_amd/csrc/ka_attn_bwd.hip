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
#include <algorithm>

#include "ka_attn.h"

namespace ssd {
namespace {

constexpr int kQueries = 128;

template <typename T>
struct AttnBwdIn {
    const T *q, *k, *v, *y, *dy;
    const float *lse;
    const int32_t *lengths;
    T *dq, *dk, *dv;
    float *delta, *partials;
    HeadStrides qs, ks, vs, ys, dys;
    int L, heads, kvheads, tiles;
    int window, sinks;
    int sink_tiles, chunk, nchunks;
    int64_t rows;  // of partial sums
    float scale, c;
};

__device__ __forceinline__ int length_of(const int32_t *lengths, int b, int L) {
    return lengths == nullptr ? L : min(max(lengths[b], 0), L);
}

template <typename T, int D>
__device__ __forceinline__ float row_dot(const T *a, const T *b) {
    float s = 0.f;
    for (int e = 0; e < D; ++e) s = fmaf(widen(a[e]), widen(b[e]), s);
    return s;
}

template <typename T, int D>
__global__ __launch_bounds__(256, 2) void attn_dq_kernel(const AttnBwdIn<T> a) {
    constexpr int KT = sizeof(T) == 2 ? 64 : 32, KB = KT / 32, NS = D / 16, DB = D / 32;
    typedef Tile<T, D, KT> Tl;
    extern __shared__ __align__(16) unsigned char lds[];

    const int group = a.heads / a.kvheads;
    int n = xcd_remap((int)blockIdx.x, (int)gridDim.x);
    const int gh = n % group;
    n /= group;
    const int q0 = (a.tiles - 1 - n % a.tiles) * kQueries;
    n /= a.tiles;
    const int kvh = n % a.kvheads, b = n / a.kvheads, head = kvh * group + gh;
    const int len = length_of(a.lengths, b, a.L);
    const int lane = threadIdx.x & 63, col = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int t = q0 + 32 * wave + col;
    const bool live = t < len;
    const int64_t dense = ((int64_t)b * a.L + t) * a.heads * D + (int64_t)head * D;
    const int64_t stat = ((int64_t)b * a.heads + head) * a.L + t;
    if (q0 >= len) {
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
    if (live && h == 0) a.delta[stat] = delta;
    const float lse = live ? a.lse[stat] * kLog2e : 0.f;

    const int t1 = min(q0 + kQueries, len) - 1;
    const int from = max(q0 - a.window + 1, 0) / KT * KT, sunk = min(a.sinks, from);
    const int nsink = (sunk + KT - 1) / KT, ntiles = nsink + (t1 - from) / KT + 1;
    const T *kh = a.k + (int64_t)b * a.ks.batch + kvh * a.ks.head, *vh = a.v + (int64_t)b * a.vs.batch + kvh * a.vs.head;
    const auto start_of = [&](int n) { return n < nsink ? n * KT : from + (n - nsink) * KT; };
    const auto stage = [&](int n) {
        const int j0 = start_of(n), rows = min((n < nsink ? sunk : len) - j0, KT);
        const uint32_t kl = lds_addr(lds + (n & 1) * 2 * Tl::kBytes);
        Tl::template copy<256>(kl, (const unsigned char *)(kh + (int64_t)j0 * a.ks.row), a.ks.row * (int64_t)sizeof(T), rows);
        Tl::template copy<256>(kl + Tl::kBytes, (const unsigned char *)(vh + (int64_t)j0 * a.vs.row), a.vs.row * (int64_t)sizeof(T), rows);
    };

    floatx16 o[DB];
#pragma unroll
    for (int db = 0; db < DB; ++db) o[db] = zero16();
    const int w0 = q0 + 32 * wave, w1 = min(w0 + 31, len - 1);
    const bool alone = t == 0 || (a.window == 1 && a.sinks == 0);  // (such a row's tile is never whole)
    stage(0);
    for (int n = 0; n < ntiles; ++n) {
        lds_dma_wait();
        __syncthreads();
        if (n + 1 < ntiles) stage(n + 1);
        const int j0 = start_of(n);
        if (w0 >= len || j0 > w1) continue;
        if (n >= nsink && j0 + KT <= w0 - a.window + 1 && j0 >= a.sinks) continue;
        const unsigned char *kl = lds + (n & 1) * 2 * Tl::kBytes, *vl = kl + Tl::kBytes;
        const bool whole = n < nsink ? j0 + KT <= sunk
                                     : j0 + KT - 1 <= w0 && (w0 + 31 - j0 < a.window || j0 + KT <= a.sinks);
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            floatx16 s = zero16(), g = zero16();
#pragma unroll
            for (int ks = 0; ks < NS; ++ks) {
                Frag<T> kf, vf;
                Tl::down(kl, 32 * kb, ks, lane, kf);
                s = mma(kf, qf[ks], s);
                Tl::down(vl, 32 * kb, ks, lane, vf);
                g = mma(vf, df[ks], g);
            }
            float ds[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) ds[r] = fast_exp2(fmaf(s[r], a.c, -lse)) * (g[r] - delta);
            if (!whole) {
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int j = j0 + 32 * kb + 8 * (r / 4) + 4 * h + r % 4;
                    ds[r] = (n < nsink ? j < sunk : sees(t, j, a.window, a.sinks)) && !alone ? ds[r] : 0.f;
                }
            }
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                Frag<T> sf;
                to_frag(ds, ks, sf);
#pragma unroll
                for (int db = 0; db < DB; ++db) {
                    Frag<T> kf;
                    Tl::across(kl, 32 * kb + 16 * ks, 32 * db, lane, kf);
                    o[db] = mma(kf, sf, o[db]);
                }
            }
        }
    }
    if (w0 >= a.L) return;  // (no barrier follows)

    float check = 0.f;
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
    // As in the forward pass: rows that a value they do not see may have spoiled, once more from what they see.
    check = both_halves(check);
    uint64_t again = __ballot(live && check != check && delta - delta == 0.f && lse - lse == 0.f) & 0xffffffffull;
    while (again != 0) {
        const int c = __builtin_ctzll(again);
        again &= again - 1;
        const int tt = w0 + c;
        const float rd = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(delta), c));
        const float rl = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(lse), c));
        const T *qr = a.q + (int64_t)b * a.qs.batch + (int64_t)tt * a.qs.row + head * a.qs.head;
        const T *dr = a.dy + (int64_t)b * a.dys.batch + (int64_t)tt * a.dys.row + head * a.dys.head;
        float acc[(D + 63) / 64] = {};
        const int near = max(tt - a.window + 1, 0), far = min(a.sinks, near), seen = far + tt - near + 1;
        for (int base = 0; base < seen; base += 64) {
            const int at = base + lane, j = at < far ? at : near + at - far;
            float ds = 0.f;
            if (at < seen && seen > 1)
                ds = fast_exp2(fmaf(row_dot<T, D>(qr, kh + (int64_t)j * a.ks.row), a.c, -rl)) *
                     (row_dot<T, D>(dr, vh + (int64_t)j * a.vs.row) - rd);
            for (int u = 0; u < min(64, seen - base); ++u) {
                const float du = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(ds), u));
                const T *kr = kh + (int64_t)(base + u < far ? base + u : near + base + u - far) * a.ks.row;
#pragma unroll
                for (int k = 0; k < (D + 63) / 64; ++k)
                    if (lane + 64 * k < D) acc[k] = fmaf(du, widen(kr[lane + 64 * k]), acc[k]);
            }
        }
        T *out = a.dq + ((int64_t)b * a.L + tt) * a.heads * D + (int64_t)head * D;
#pragma unroll
        for (int k = 0; k < (D + 63) / 64; ++k)
            if (lane + 64 * k < D) narrow(out + lane + 64 * k, acc[k] * a.scale);
    }
}

// 128 keys, 32 a wave in registers (columns of the products S = Q K^T, dP = dY
// V^T), against tiles of 32 queries; dv^T += dY^T P and dk^T += Q^T dS take the
// same tiles across.
template <typename T, int D>
__global__ __launch_bounds__(256, 1) void attn_dkv_kernel(const AttnBwdIn<T> a) {
    constexpr int NS = D / 16, DB = D / 32;
    typedef Tile<T, D, 32> Tl;
    extern __shared__ __align__(16) unsigned char lds[];  // (2 stages, queries and dy), then (2 stages, lse and delta)
    float *stats = reinterpret_cast<float *>(lds + 4 * Tl::kBytes);

    const int group = a.heads / a.kvheads, ntiles = (a.L + kAttnKeys - 1) / kAttnKeys;
    const int items = ntiles + a.sink_tiles * a.nchunks;
    int n = xcd_remap((int)blockIdx.x, (int)gridDim.x);
    const int item = n % items;
    n /= items;
    const int kvh = n % a.kvheads, b = n / a.kvheads;
    const int len = length_of(a.lengths, b, a.L);
    // a tile's queries through the window, or a chunk of those that see its sinks from farther
    const bool sunk = item >= ntiles;
    const int tile = sunk ? (item - ntiles) / a.nchunks : item, part = sunk ? 1 + (item - ntiles) % a.nchunks : 0;
    const int j0 = tile * kAttnKeys;
    int lo = j0, hi = (int)min((int64_t)len, (int64_t)j0 + kAttnKeys - 1 + a.window);
    if (sunk) {
        lo = max(a.window + (part - 1) * a.chunk, a.window + j0);
        hi = min(len, a.window + part * a.chunk);
    }
    const int nq = hi > lo ? (hi - lo + 31) / 32 : 0, turns = nq * group;

    const int lane = threadIdx.x & 63, col = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int w0 = j0 + 32 * wave, j = w0 + col;
    const bool live = j < len;
    const T *kh = a.k + (int64_t)b * a.ks.batch + kvh * a.ks.head, *vh = a.v + (int64_t)b * a.vs.batch + kvh * a.vs.head;
    const T *qb = a.q + (int64_t)b * a.qs.batch, *db_ = a.dy + (int64_t)b * a.dys.batch;
    Frag<T> kf[NS], vf[NS];
#pragma unroll
    for (int s = 0; s < NS; ++s) {
        load_frag(kf[s], kh + (int64_t)j * a.ks.row + 16 * s + 8 * h, live);
        load_frag(vf[s], vh + (int64_t)j * a.vs.row + 16 * s + 8 * h, live);
    }

    const auto stage = [&](int n) {
        const int head = kvh * group + n / nq, t0 = lo + n % nq * 32, rows = min(hi - t0, 32);
        const uint32_t ql = lds_addr(lds + (n & 1) * 2 * Tl::kBytes);
        Tl::template copy<256>(ql, (const unsigned char *)(qb + (int64_t)t0 * a.qs.row + head * a.qs.head), a.qs.row * (int64_t)sizeof(T), rows);
        Tl::template copy<256>(ql + Tl::kBytes, (const unsigned char *)(db_ + (int64_t)t0 * a.dys.row + head * a.dys.head),
                               a.dys.row * (int64_t)sizeof(T), rows);
        if (threadIdx.x < 64) {
            const int64_t at = ((int64_t)b * a.heads + head) * a.L + t0 + col;
            float s = 0.f;
            if (col < rows) s = h == 0 ? a.lse[at] * kLog2e : a.delta[at];
            stats[(n & 1) * 64 + h * 32 + col] = s;
        }
    };

    const bool lone = a.window == 1 && a.sinks == 0;
    floatx16 dk[DB], dv[DB];
#pragma unroll
    for (int db = 0; db < DB; ++db) dk[db] = dv[db] = zero16();
    if (turns > 0) stage(0);
    for (int n = 0; n < turns; ++n) {
        lds_dma_wait();
        __syncthreads();
        if (n + 1 < turns) stage(n + 1);
        const int t0 = lo + n % nq * 32;
        if (sunk ? w0 >= a.sinks || t0 + 31 - w0 < a.window : t0 + 31 < w0 || t0 - w0 - 31 >= a.window) continue;
        const bool whole = sunk ? w0 + 32 <= a.sinks && t0 - w0 - 31 >= 0 && t0 - w0 - 31 >= a.window
                                : t0 >= w0 + 31 && t0 + 31 - w0 < a.window;
        const unsigned char *ql = lds + (n & 1) * 2 * Tl::kBytes, *dl = ql + Tl::kBytes;
        floatx16 s = zero16(), g = zero16();
#pragma unroll
        for (int ks = 0; ks < NS; ++ks) {
            Frag<T> f;
            Tl::down(ql, 0, ks, lane, f);
            s = mma(f, kf[ks], s);
            Tl::down(dl, 0, ks, lane, f);
            g = mma(f, vf[ks], g);
        }
        float p[16], ds[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int row = 8 * (r / 4) + 4 * h + r % 4;
            p[r] = fast_exp2(fmaf(s[r], a.c, -stats[(n & 1) * 64 + row]));
            ds[r] = p[r] * (g[r] - stats[(n & 1) * 64 + 32 + row]);
        }
        if (!whole) {
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int t = t0 + 8 * (r / 4) + 4 * h + r % 4;
                const bool on = t < hi && (sunk ? j < a.sinks && t - j >= a.window : j <= t && t - j < a.window);
                p[r] = on ? p[r] : 0.f;
                ds[r] = on && t > 0 && !lone ? ds[r] : 0.f;
            }
        }
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            Frag<T> pf, sf;
            to_frag(p, ks, pf);
            to_frag(ds, ks, sf);
#pragma unroll
            for (int db = 0; db < DB; ++db) {
                Frag<T> f;
                Tl::across(dl, 16 * ks, 32 * db, lane, f);
                dv[db] = mma(f, pf, dv[db]);
                Tl::across(ql, 16 * ks, 32 * db, lane, f);
                dk[db] = mma(f, sf, dk[db]);
            }
        }
    }

    const bool partial = tile < a.sink_tiles;
    const int64_t dense = ((int64_t)b * a.L + j) * a.kvheads * D + (int64_t)kvh * D;
    float *pk = a.partials + ((((int64_t)b * a.kvheads + kvh) * (1 + a.nchunks) + part) * 2 * a.rows + j) * D;
    float *pv = pk + a.rows * D;
    float check = 0.f;
#pragma unroll
    for (int db = 0; db < DB; ++db) {
        float x[16], z[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            check = fmaf(dk[db][r], 0.f, fmaf(dv[db][r], 0.f, check));
            x[r] = live ? dk[db][r] * a.scale : 0.f;
            z[r] = live ? dv[db][r] : 0.f;
        }
        if (partial) {
            store_column(pk, db, h, x, true);
            store_column(pv, db, h, z, true);
        } else {
            store_column(a.dk + dense, db, h, x, j < a.L);
            store_column(a.dv + dense, db, h, z, j < a.L);
        }
    }
    // Keys that a query which does not see them may have spoiled, once more from those that do.
    check = both_halves(check);
    uint64_t again = __ballot(live && check != check) & 0xffffffffull;
    while (again != 0) {
        const int c = __builtin_ctzll(again);
        again &= again - 1;
        const int jj = w0 + c;
        const T *kr = kh + (int64_t)jj * a.ks.row, *vr = vh + (int64_t)jj * a.vs.row;
        const int t_lo = sunk ? max(lo, jj + a.window) : jj, t_hi = sunk ? (jj < a.sinks ? hi : t_lo) : (int)min((int64_t)hi, (int64_t)jj + a.window);
        float acc[2][(D + 63) / 64] = {};
        for (int gh = 0; gh < group; ++gh) {
            const int head = kvh * group + gh;
            for (int base = t_lo; base < t_hi; base += 64) {
                const int t = base + lane;
                float p = 0.f, ds = 0.f;
                if (t < t_hi) {
                    const int64_t at = ((int64_t)b * a.heads + head) * a.L + t;
                    p = fast_exp2(fmaf(row_dot<T, D>(qb + (int64_t)t * a.qs.row + head * a.qs.head, kr), a.c, -a.lse[at] * kLog2e));
                    if (t > 0 && !lone)
                        ds = p * (row_dot<T, D>(db_ + (int64_t)t * a.dys.row + head * a.dys.head, vr) - a.delta[at]);
                }
                for (int u = 0; u < min(64, t_hi - base); ++u) {
                    const float pu = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(p), u));
                    const float su = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(ds), u));
                    const T *qr = qb + (int64_t)(base + u) * a.qs.row + head * a.qs.head;
                    const T *dr = db_ + (int64_t)(base + u) * a.dys.row + head * a.dys.head;
#pragma unroll
                    for (int k = 0; k < (D + 63) / 64; ++k)
                        if (lane + 64 * k < D) {
                            acc[0][k] = fmaf(su, widen(qr[lane + 64 * k]), acc[0][k]);
                            acc[1][k] = fmaf(pu, widen(dr[lane + 64 * k]), acc[1][k]);
                        }
                }
            }
        }
        const int64_t out = ((int64_t)b * a.L + jj) * a.kvheads * D + (int64_t)kvh * D;
        float *qk = a.partials + ((((int64_t)b * a.kvheads + kvh) * (1 + a.nchunks) + part) * 2 * a.rows + jj) * D;
#pragma unroll
        for (int k = 0; k < (D + 63) / 64; ++k) {
            const int e = lane + 64 * k;
            if (e >= D) continue;
            if (partial) {
                qk[e] = acc[0][k] * a.scale;
                qk[a.rows * D + e] = acc[1][k];
            } else {
                narrow(a.dk + out + e, acc[0][k] * a.scale);
                narrow(a.dv + out + e, acc[1][k]);
            }
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
        for (int k = 0; k < parts; ++k) s += p[k * 2 * a.rows * D];
        narrow((second ? a.dv : a.dk) + ((b * a.L + j) * a.kvheads + kvh) * D + e, s);
    }
}

template <typename T, int D>
hipError_t attn_bwd_sized(const AttnBwdIn<T> &in, int64_t batch, hipStream_t stream) {
    constexpr int kLdsQ = 2 * 2 * Tile<T, D, sizeof(T) == 2 ? 64 : 32>::kBytes, kLdsK = 2 * 2 * Tile<T, D, 32>::kBytes + 2 * 2 * 32 * (int)sizeof(float);
    hipError_t e = allow_lds<attn_dq_kernel<T, D>>(kLdsQ);
    if (e == hipSuccess) e = allow_lds<attn_dkv_kernel<T, D>>(kLdsK);
    if (e != hipSuccess) return e;
    attn_dq_kernel<T, D><<<dim3((uint32_t)(batch * in.heads * in.tiles)), dim3(256), kLdsQ, stream>>>(in);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    const int64_t items = (in.L + kAttnKeys - 1) / kAttnKeys + (int64_t)in.sink_tiles * in.nchunks;
    attn_dkv_kernel<T, D><<<dim3((uint32_t)(batch * in.kvheads * items)), dim3(256), kLdsK, stream>>>(in);
    if ((e = hipGetLastError()) != hipSuccess || in.sink_tiles == 0) return e;
    const int64_t heads = batch * in.kvheads, n = 2 * heads * std::min<int64_t>(in.L, in.rows) * D;
    attn_sinks_kernel<T><<<dim3((uint32_t)std::min<int64_t>((n + 255) / 256, 1 << 16)), dim3(256), 0, stream>>>(in, heads, D);
    return hipGetLastError();
}

template <typename T>
hipError_t attn_bwd_typed(const AttnArgs &a, const AttnBwdPlan &p, hipStream_t stream) {
    const AttnBwdIn<T> in{static_cast<const T *>(a.q), static_cast<const T *>(a.k), static_cast<const T *>(a.v),
                          static_cast<const T *>(a.y), static_cast<const T *>(a.dy), a.lse, a.lengths,
                          static_cast<T *>(a.dq), static_cast<T *>(a.dk), static_cast<T *>(a.dv), a.delta, a.partials,
                          a.qs, a.ks, a.vs, a.ys, a.dys, a.seqlen, a.heads, a.kvheads, (a.seqlen + kQueries - 1) / kQueries,
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
