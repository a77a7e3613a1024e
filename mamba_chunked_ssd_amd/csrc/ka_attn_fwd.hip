// ka_attn_fwd.hip -- sliding-window attention with sinks over prompts.
//
//   s_tj = scale q_t . k_j ,  y_t = sum_j exp(s_tj - lse_t) v_j  over the keys
//   that t sees: the last `window` tokens and the first `sinks`.
//
// One pass over the keys with the running maximum and sum of the softmax.  A
// wave owns 32 queries, a block of four 128; tiles of keys and values come into
// LDS by asynchronous copies, one tile ahead.  The products are S^T = K Q^T and
// O^T = V^T P^T, so that a query is a lane's column throughout: its maximum, sum
// and rescaling are the lane's own but for one exchange of the two halves, and P
// stays in registers as the second product's operand.
#include <algorithm>
#include <limits>

#include "ka_attn.h"

namespace ssd {
namespace {

constexpr float kInf = std::numeric_limits<float>::infinity();
constexpr int kQueries = 128;  // of a block

template <typename T>
struct AttnIn {
    const T *q, *k, *v;
    T *kc, *vc;
    const int32_t *positions, *lengths;
    T *y;
    float *lse;
    HeadStrides qs, ks, vs;
    int64_t slots;  // of the cache
    int L, heads, kvheads, tiles;
    int window, sinks;
    float c;  // scale log2(e)
};

// The keys of one sequence and head: new ones, and the cache's of the tokens before `first`.
template <typename T, int D>
struct Keys {
    const T *fresh, *cache;
    int64_t row;
    int first, window, sinks;
    __device__ const T *of(int j) const {
        if (j >= first) return fresh + (int64_t)(j - first) * row;
        return cache + (int64_t)(j < sinks ? j : sinks + (j - sinks) % window) * D;
    }
};

template <typename T, int D>
__global__ __launch_bounds__(256, 2) void attn_fwd_kernel(const AttnIn<T> a) {
    constexpr int KT = sizeof(T) == 2 ? 64 : 32, KB = KT / 32, NS = D / 16, DB = D / 32;
    typedef Tile<T, D, KT> Tl;
    extern __shared__ __align__(16) unsigned char lds[];  // (2 stages, keys and values)

    const int group = a.heads / a.kvheads;
    int n = xcd_remap((int)blockIdx.x, (int)gridDim.x);
    const int gh = n % group;
    n /= group;
    const int q0 = (a.tiles - 1 - n % a.tiles) * kQueries;  // the longest rows of keys first
    n /= a.tiles;
    const int kvh = n % a.kvheads, b = n / a.kvheads, head = kvh * group + gh;
    const int len = a.lengths == nullptr ? a.L : min(max(a.lengths[b], 0), a.L);
    const int first = a.positions == nullptr ? 0 : min(max(a.positions[b], 0), kAttnLast);
    const int end = first + len;

    const int lane = threadIdx.x & 63, col = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int i = q0 + 32 * wave + col, t = first + i;
    const bool live = i < len;
    T *yrow = a.y + ((int64_t)b * a.L + i) * a.heads * D + (int64_t)head * D;
    float *lse = a.lse != nullptr ? a.lse + ((int64_t)b * a.heads + head) * a.L + i : nullptr;
    if (q0 >= len) {
        if (i < a.L) {
            const float z[16] = {};
            for (int db = 0; db < DB; ++db) store_column(yrow, db, h, z, true);
            if (lse != nullptr && h == 0) *lse = 0.f;
        }
        return;
    }

    Frag<T> qf[NS];
    const T *qrow = a.q + (int64_t)b * a.qs.batch + (int64_t)i * a.qs.row + head * a.qs.head;
#pragma unroll
    for (int s = 0; s < NS; ++s) load_frag(qf[s], qrow + 16 * s + 8 * h, live);

    // Tiles of keys: those of the window from `from`, on a grid that `first` lies on, and before them the sinks
    // below `from`.
    const int t0 = first + q0, t1 = min(t0 + kQueries, end) - 1;
    const int lo = max(t0 - a.window + 1, 0);
    const int from = lo >= first ? first + (lo - first) / KT * KT : first - (first - lo + KT - 1) / KT * KT;
    const int sunk = min(a.sinks, max(from, 0));
    const int nsink = (sunk + KT - 1) / KT, ntiles = nsink + (t1 - from) / KT + 1;
    const Keys<T, D> keys{a.k + (int64_t)b * a.ks.batch + kvh * a.ks.head, a.kc + ((int64_t)b * a.kvheads + kvh) * a.slots * D,
                          a.ks.row, first, a.window, a.sinks};
    const Keys<T, D> values{a.v + (int64_t)b * a.vs.batch + kvh * a.vs.head,
                            a.vc + ((int64_t)b * a.kvheads + kvh) * a.slots * D, a.vs.row, first, a.window, a.sinks};
    const auto start_of = [&](int n) { return n < nsink ? n * KT : from + (n - nsink) * KT; };
    const auto stage = [&](int n) {
        const int j0 = start_of(n), stop = n < nsink ? sunk : end;
        unsigned char *kl = lds + (n & 1) * 2 * Tl::kBytes, *vl = kl + Tl::kBytes;
        if (j0 >= first) {
            const int rows = min(stop - j0, KT);
            Tl::template copy<256>(lds_addr(kl), (const unsigned char *)(keys.fresh + (int64_t)(j0 - first) * a.ks.row),
                                   a.ks.row * (int64_t)sizeof(T), rows);
            Tl::template copy<256>(lds_addr(vl), (const unsigned char *)(values.fresh + (int64_t)(j0 - first) * a.vs.row),
                                   a.vs.row * (int64_t)sizeof(T), rows);
        } else {
            // the cache holds what some query of this call may see, and no older token
            const auto held = [&](int j) { return j >= 0 && j < stop && (n < nsink || j >= lo || j < a.sinks); };
            Tl::template gather<256>(kl, [&](int r) { return held(j0 + r) ? keys.of(j0 + r) : nullptr; });
            Tl::template gather<256>(vl, [&](int r) { return held(j0 + r) ? values.of(j0 + r) : nullptr; });
        }
    };

    floatx16 o[DB];
#pragma unroll
    for (int db = 0; db < DB; ++db) o[db] = zero16();
    float m = -kInf, l = 0.f;  // in units of log 2; l of this lane's half of the keys
    const int w0 = t0 + 32 * wave, w1 = min(w0 + 31, end - 1);  // the wave's queries

    stage(0);
    for (int n = 0; n < ntiles; ++n) {
        lds_dma_wait();
        __syncthreads();
        if (n + 1 < ntiles) stage(n + 1);
        const int j0 = start_of(n);
        if (w0 >= end || j0 > w1) continue;
        if (n >= nsink && j0 + KT <= w0 - a.window + 1 && j0 >= a.sinks) continue;
        const unsigned char *kl = lds + (n & 1) * 2 * Tl::kBytes, *vl = kl + Tl::kBytes;
        floatx16 s[KB];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            s[kb] = zero16();
#pragma unroll
            for (int ks = 0; ks < NS; ++ks) {
                Frag<T> kf;
                Tl::down(kl, 32 * kb, ks, lane, kf);
                s[kb] = mma(kf, qf[ks], s[kb]);
            }
        }
        const bool whole = n < nsink ? j0 + KT <= sunk
                                     : j0 >= 0 && j0 + KT - 1 <= w0 && (w0 + 31 - j0 < a.window || j0 + KT <= a.sinks);
        if (!whole) {
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int j = j0 + 32 * kb + 8 * (r / 4) + 4 * h + r % 4;
                    const bool on = n < nsink ? j < sunk : j >= 0 && sees(t, j, a.window, a.sinks);
                    s[kb][r] = on ? s[kb][r] : -kInf;
                }
        }
        float top = s[0][0];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int r = 0; r < 16; ++r) top = fmaxf(top, s[kb][r]);
        top = fmaxf(top, other_half(top)) * a.c;
        // The reference of the exponentials follows the maximum only where it has fallen 2^8 behind: p stays below
        // 2^8, which costs no precision, and most tiles rescale nothing.
        if (__any(top > m + 8.f)) {
            const float next = fmaxf(m, top);
            const float by = next == -kInf ? 1.f : fast_exp2(m - next);
            l *= by;
#pragma unroll
            for (int db = 0; db < DB; ++db)
#pragma unroll
                for (int r = 0; r < 16; ++r) o[db][r] *= by;
            m = next;
        }
        const float ref = m == -kInf ? 0.f : m;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            float p[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                p[r] = fast_exp2(fmaf(s[kb][r], a.c, -ref));
                l += p[r];
            }
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                Frag<T> pf;
                to_frag(p, ks, pf);
#pragma unroll
                for (int db = 0; db < DB; ++db) {
                    Frag<T> vf;
                    Tl::across(vl, 32 * kb + 16 * ks, 32 * db, lane, vf);
                    o[db] = mma(vf, pf, o[db]);
                }
            }
        }
    }
    if (w0 - first >= a.L) return;  // (no barrier follows)

    l = both_halves(l);
    const float ref = m == -kInf ? 0.f : m, inv = 1.f / l;
    float check = 0.f;  // NaN if a sum is not finite
#pragma unroll
    for (int db = 0; db < DB; ++db) {
        float v[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            check = fmaf(o[db][r], 0.f, check);
            v[r] = live ? o[db][r] * inv : 0.f;
        }
        store_column(yrow, db, h, v, i < a.L);
    }
    if (lse != nullptr && h == 0 && i < a.L) *lse = live ? (m + __builtin_amdgcn_logf(l)) * 0.6931471805599453f : 0.f;

    // A value that is not finite makes 0 times it NaN in the rows of its tile that do not see it.  Such rows (with
    // a sound softmax) are formed again, each from the tokens that it sees alone: 64 keys' weights at a time, a lane
    // each, then their values one after the other, a lane to an element.
    check = both_halves(check);
    uint64_t again = __ballot(live && check != check && l > 0.f && l < kInf) & 0xffffffffull;
    while (again != 0) {
        const int c = __builtin_ctzll(again);
        again &= again - 1;
        const int tt = w0 + c;
        const float rm = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(ref), c));
        const float rl = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(inv), c));
        const T *qr = a.q + (int64_t)b * a.qs.batch + (int64_t)(tt - first) * a.qs.row + head * a.qs.head;
        float acc[(D + 63) / 64] = {};
        const int near = max(tt - a.window + 1, 0), far = min(a.sinks, near), seen = far + tt - near + 1;
        for (int base = 0; base < seen; base += 64) {
            const int at = base + lane, j = at < far ? at : near + at - far;
            float p = 0.f;
            if (at < seen) {
                const T *kr = keys.of(j);
                float s = 0.f;
                for (int e = 0; e < D; ++e) s = fmaf(widen(qr[e]), widen(kr[e]), s);
                p = fast_exp2(fmaf(s, a.c, -rm));
            }
            for (int u = 0; u < min(64, seen - base); ++u) {
                const float pu = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(p), u));
                const int ju = base + u < far ? base + u : near + base + u - far;
                const T *vr = values.of(ju);
#pragma unroll
                for (int k = 0; k < (D + 63) / 64; ++k)
                    if (lane + 64 * k < D) acc[k] = fmaf(pu, widen(vr[lane + 64 * k]), acc[k]);
            }
        }
        T *yr = a.y + ((int64_t)b * a.L + (tt - first)) * a.heads * D + (int64_t)head * D;
#pragma unroll
        for (int k = 0; k < (D + 63) / 64; ++k)
            if (lane + 64 * k < D) narrow(yr + lane + 64 * k, acc[k] * rl);
    }
}

// The new tokens that stay in the cache: the first `sinks` and the last
// `window` of a sequence.  A thread copies 16 bytes of a key and of a value.
template <typename T>
__global__ __launch_bounds__(256) void attn_put_kernel(const AttnIn<T> a, int D, int front, int rows) {
    const int b = blockIdx.y, pieces = D * (int)sizeof(T) / 16, per = 16 / (int)sizeof(T);
    const int len = a.lengths == nullptr ? a.L : min(max(a.lengths[b], 0), a.L);
    const int first = a.positions == nullptr ? 0 : min(max(a.positions[b], 0), kAttnLast);
    const int64_t all = (int64_t)rows * a.kvheads * pieces;
    for (int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x; n < all; n += (int64_t)gridDim.x * 256) {
        const int piece = (int)(n % pieces);
        const int64_t rest = n / pieces;
        const int head = (int)(rest % a.kvheads), row = (int)(rest / a.kvheads);
        // rows 0 .. front - 1: tokens that may be sinks; then those of the window, the last first
        const int i = row < front ? row : len - 1 - (row - front), j = first + i;
        if (i < 0 || i >= len || (row < front) != (j < a.sinks)) continue;
        const int64_t slot = j < a.sinks ? j : a.sinks + (j - a.sinks) % a.window;
        const int64_t to = (((int64_t)b * a.kvheads + head) * a.slots + slot) * D + piece * per;
        *reinterpret_cast<u32x4 *>(a.kc + to) = *reinterpret_cast<const u32x4 *>(a.k + b * a.ks.batch + i * a.ks.row + head * a.ks.head + piece * per);
        *reinterpret_cast<u32x4 *>(a.vc + to) = *reinterpret_cast<const u32x4 *>(a.v + b * a.vs.batch + i * a.vs.row + head * a.vs.head + piece * per);
    }
}

template <typename T, int D>
hipError_t attn_fwd_sized(const AttnIn<T> &in, int64_t batch, hipStream_t stream) {
    constexpr int kLds = 2 * 2 * Tile<T, D, sizeof(T) == 2 ? 64 : 32>::kBytes;
    const hipError_t e = allow_lds<attn_fwd_kernel<T, D>>(kLds);
    if (e != hipSuccess) return e;
    attn_fwd_kernel<T, D><<<dim3((uint32_t)(batch * in.heads * in.tiles)), dim3(256), kLds, stream>>>(in);
    return hipGetLastError();
}

template <typename T>
hipError_t attn_fwd_typed(const AttnArgs &a, hipStream_t stream) {
    const AttnIn<T> in{static_cast<const T *>(a.q), static_cast<const T *>(a.k), static_cast<const T *>(a.v),
                       static_cast<T *>(a.kc), static_cast<T *>(a.vc), a.positions, a.lengths, static_cast<T *>(a.y), a.lse,
                       a.qs, a.ks, a.vs, (int64_t)a.window + a.sinks, a.seqlen, a.heads, a.kvheads,
                       (a.seqlen + kQueries - 1) / kQueries, a.window, a.sinks, a.scale * kLog2e};
    hipError_t e = a.headdim == 32   ? attn_fwd_sized<T, 32>(in, a.batch, stream)
                   : a.headdim == 64 ? attn_fwd_sized<T, 64>(in, a.batch, stream)
                                     : attn_fwd_sized<T, 128>(in, a.batch, stream);
    if (e != hipSuccess || a.kc == nullptr) return e;
    // after the attention, which reads what these rows replace
    const int front = std::min(a.sinks, a.seqlen), rows = front + std::min(a.window, a.seqlen);
    const int64_t pieces = (int64_t)rows * a.kvheads * (a.headdim * (int)sizeof(T) / 16);
    attn_put_kernel<T><<<dim3((uint32_t)std::min<int64_t>((pieces + 255) / 256, 1 << 12), (uint32_t)a.batch), dim3(256), 0, stream>>>(
        in, a.headdim, front, rows);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_fwd(const AttnArgs &a, hipStream_t stream) {
    return a.bf16 ? attn_fwd_typed<uint16_t>(a, stream) : attn_fwd_typed<float>(a, stream);
}

}  // namespace ssd
