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
//
// Bound by the waves' own chain of products, exponentials and waits at two (heads
// of 128) or three (64) waves to a SIMD.  16 384 tokens, 8 heads of 128 over 2, a
// window of 2048: 153 to 166 us, 780 to 847 TFLOP/s (an 8192^3 product of the
// library: 1170); alone on its SIMD a wave takes 218.  2 x 2048 tokens, 40 heads of
// 64 over 8, a window of 512: 40 us (one, two, three blocks to a compute unit: 77,
// 49, 40).  LDS is no limit: its pipe is busy 17 % of the time, without conflicts.
#include <algorithm>

#include "ka_attn.h"

namespace ssd {
namespace {

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
    int L, heads, kvheads;
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

// What a lane's query t, one of the wave's from w0 on, does not see of 32 KB keys from token j0, of tile n, becomes
// -infinity.
template <int KT, int KB>
__device__ __forceinline__ void hide(floatx16 (&s)[KB], const Walk<KT> &w, int n, int j0, int t, int w0, int h, int window, int sinks) {
    const Needs need(j0, 32 * KB, w0, window, sinks);
    const Mask mask(t, j0, h, window, sinks);
    if (n < w.nsink) {
        const int sunk = w.sunk - j0 - 4 * h;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int r = 0; r < 16; ++r) s[kb][r] = place(kb, r) < sunk ? s[kb][r] : -kInf;
    } else if (!need.before) {
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int r = 0; r < 16; ++r) s[kb][r] = place(kb, r) <= mask.last ? s[kb][r] : -kInf;
    } else if (!need.last && j0 >= sinks) {
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int r = 0; r < 16; ++r) s[kb][r] = place(kb, r) > mask.before ? s[kb][r] : -kInf;
    } else {
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int r = 0; r < 16; ++r) s[kb][r] = mask.seen(place(kb, r)) ? s[kb][r] : -kInf;
    }
    if (j0 < 0) {
        const int none = -j0 - 4 * h;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int r = 0; r < 16; ++r) s[kb][r] = place(kb, r) >= none ? s[kb][r] : -kInf;
    }
}

// Elements 32 db .. of a wave's rows formed again (see with_odd): queries w0 ..
// w0 + 31 below `end`, a lane's t with its softmax's reference and 1 / sum, over
// the sinks and the window's tokens, 32 at a time.  A score of -infinity has a
// weight of 0, which makes NaN of a value that is not finite.
template <typename T, int D>
__device__ __forceinline__ void attend_again(const AttnIn<T> &a, const Keys<T, D> &keys, const Keys<T, D> &values,
                                             const Frag<T> (&q)[D / 16], int w0, int end, int t, int db, float ref, float inv,
                                             T *row, bool on) {
    const int lane = threadIdx.x & 63, col = lane & 31, h = lane >> 5;
    const int near = max(w0 - a.window + 1, 0), last = min(w0 + 31, end - 1), far = min(a.sinks, near);
    const int nfar = (far + 31) / 32, blocks = nfar + (last - near) / 32 + 1;
    floatx16 o = zero16();
    uint32_t odd = 0;
#pragma unroll 1
    for (int n = 0; n < blocks; ++n) {
        const int j0 = n < nfar ? 32 * n : near + 32 * (n - nfar), stop = n < nfar ? far : last + 1;
        floatx16 s = zero16(), kinds = zero16();
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            Frag<T> kf;
            load_frag(kf, keys.of(j0 + col) + 16 * ks + 8 * h, j0 + col < stop);
            s = mma(kf, q[ks], s);
        }
        const int upto = min(t, stop - 1) - j0 - 4 * h, before = t - a.window - j0 - 4 * h, sunk = a.sinks - j0 - 4 * h;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            float p[8], u[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = 8 * ks + i, at = place(0, r);
                const bool seen = (at <= upto) & ((at > before) | (at < sunk));
                p[i] = seen ? fast_exp2(fmaf(s[r], a.c, -ref)) : 0.f;
                u[i] = !seen ? 0.f : s[r] == -kInf ? kOddNan : 1.f;
            }
            Frag<T> pf, uf, vf, kind;
            to_frag(p, pf);
            to_frag(u, uf);
            load_apart(vf, kind, 32 * db + col, [&](int i) {
                const int j = j0 + 16 * ks + 4 * h + i;
                return j < stop ? values.of(j) : nullptr;
            });
            o = mma(vf, pf, o);
            kinds = mma(kind, uf, kinds);
        }
        odd |= odd_of(kinds);
    }
    float v[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) v[r] = with_odd(o[r] * inv, odd, r);
    store_column(row, db, h, v, on);
}

// What a block works on.
template <typename T, int D>
struct Place {
    int head, kvh, b, q0, len, first, end;
    // queries: of a block; the longest rows of keys come first
    __device__ Place(const AttnIn<T> &a, int queries) {
        const int group = a.heads / a.kvheads, tiles = (a.L + queries - 1) / queries;
        int n = xcd_remap((int)blockIdx.x, (int)gridDim.x);
        const int gh = n % group;
        n /= group;
        q0 = (tiles - 1 - n % tiles) * queries;
        n /= tiles;
        kvh = n % a.kvheads;
        b = n / a.kvheads;
        head = kvh * group + gh;
        len = a.lengths == nullptr ? a.L : min(max(a.lengths[b], 0), a.L);
        first = a.positions == nullptr ? 0 : min(max(a.positions[b], 0), kAttnLast);
        end = first + len;
    }
    __device__ Keys<T, D> keys(const AttnIn<T> &a) const {
        return Keys<T, D>{a.k + (int64_t)b * a.ks.batch + kvh * a.ks.head, a.kc + ((int64_t)b * a.kvheads + kvh) * a.slots * D,
                          a.ks.row, first, a.window, a.sinks};
    }
    __device__ Keys<T, D> values(const AttnIn<T> &a) const {
        return Keys<T, D>{a.v + (int64_t)b * a.vs.batch + kvh * a.vs.head, a.vc + ((int64_t)b * a.kvheads + kvh) * a.slots * D,
                          a.vs.row, first, a.window, a.sinks};
    }
    __device__ const T *query(const AttnIn<T> &a, int i) const {
        return a.q + (int64_t)b * a.qs.batch + (int64_t)i * a.qs.row + head * a.qs.head;
    }
    __device__ T *result(const AttnIn<T> &a, int i) const {
        return a.y + ((int64_t)b * a.L + i) * a.heads * D + (int64_t)head * D;
    }
    __device__ float *sums(const AttnIn<T> &a, int i) const {
        return a.lse + ((int64_t)b * a.heads + head) * a.L + i;
    }
};
constexpr float kLn2 = 0.6931471805599453f;

template <typename T, int D>
__global__ __launch_bounds__(256, (sizeof(T) == 2 ? (D == 32 ? 4 : D == 64 ? 3 : 2) : (D == 128 ? 1 : 2))) void attn_fwd_kernel(const AttnIn<T> a) {
    constexpr int KT = sizeof(T) == 2 ? 64 : 32, KB = KT / 32, NS = D / 16, DB = D / 32;
    typedef Tile<T, D, KT> Tl;
    extern __shared__ __align__(16) unsigned char lds[];  // (2 stages, keys and values)

    const Place<T, D> p(a, kQueries);
    const int lane = threadIdx.x & 63, col = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int i = p.q0 + 32 * wave + col, t = p.first + i;
    const bool live = i < p.len;
    if (p.q0 >= p.len) {
        if (i < a.L) {
            const float z[16] = {};
            for (int db = 0; db < DB; ++db) store_column(p.result(a, i), db, h, z, true);
            if (a.lse != nullptr && h == 0) *p.sums(a, i) = 0.f;
        }
        return;
    }
    Frag<T> qf[NS];
#pragma unroll
    for (int s = 0; s < NS; ++s) load_frag(qf[s], p.query(a, i) + 16 * s + 8 * h, live);

    const int t0 = p.first + p.q0;
    const Walk<KT> walk(t0, min(t0 + kQueries, p.end) - 1, p.first, a.window, a.sinks);
    const Keys<T, D> keys = p.keys(a), values = p.values(a);
    Copier<Tl, 4> kcopy, vcopy;
    kcopy.init(a.ks.row * (int64_t)sizeof(T), wave, lane);
    vcopy.init(a.vs.row * (int64_t)sizeof(T), wave, lane);
    const auto stage = [&](int n) {
        const int j0 = walk.start(n);
        unsigned char *kl = lds + (n & 1) * 2 * Tl::kBytes, *vl = kl + Tl::kBytes;
        if (j0 >= p.first) {
            const int rows = min((n < walk.nsink ? walk.sunk : p.end) - j0, KT);
            kcopy.copy(lds_addr(kl), keys.of(j0), rows);
            vcopy.copy(lds_addr(vl), values.of(j0), rows);
        } else {
            Tl::template gather<256>(kl, [&](int r) { return walk.held(n, j0 + r, a.sinks, p.end) ? keys.of(j0 + r) : nullptr; });
            Tl::template gather<256>(vl, [&](int r) { return walk.held(n, j0 + r, a.sinks, p.end) ? values.of(j0 + r) : nullptr; });
        }
    };

    if (walk.ntiles > 0) stage(0);
#pragma unroll
    for (int s = 0; s < NS; ++s) arrived(qf[s]);
    Running<T, D> run;
    run.init();
    const int w0 = t0 + 32 * wave, w1 = min(w0 + 31, p.end - 1);  // the wave's queries
    for (int n = 0; n < walk.ntiles; ++n) {
        lds_dma_wait();
        __syncthreads();
        if (n + 1 < walk.ntiles) stage(n + 1);
        if (w0 >= p.end) continue;
        const unsigned char *kl = lds + (n & 1) * 2 * Tl::kBytes, *vl = kl + Tl::kBytes;
        const int j0 = walk.start(n);
        if (j0 > w1 || (n >= walk.nsink && j0 + KT <= w0 - a.window + 1 && j0 >= a.sinks)) continue;
        floatx16 s[KB];
        scores<Tl>(kl, qf, lane, s);
        const bool whole = n < walk.nsink ? j0 + KT <= walk.sunk
                                          : j0 >= 0 && j0 + KT - 1 <= w0 && (w0 + 31 - j0 < a.window || j0 + KT <= a.sinks);
        if (!whole) hide(s, walk, n, j0, t, w0, h, a.window, a.sinks);
        run.template take<Tl, KB>(s, a.c, vl, lane);
    }
    if (w0 - p.first >= a.L) return;  // (no barrier follows)

    const float l = both_halves(run.l), ref = run.ref(), inv = 1.f / l;
    float check = 0.f;  // NaN if a sum is not finite
#pragma unroll
    for (int db = 0; db < DB; ++db) {
        float v[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            check = fmaf(run.o[db][r], 0.f, check);
            v[r] = live ? run.o[db][r] * inv : 0.f;
        }
        store_column(p.result(a, i), db, h, v, i < a.L);
    }
    if (a.lse != nullptr && h == 0 && i < a.L) *p.sums(a, i) = live ? (run.m + __builtin_amdgcn_logf(l)) * kLn2 : 0.f;
    check = both_halves(check);
    const bool redo = live && check != check && l > 0.f && l < kInf;
    if (__any(redo)) {
#pragma unroll 1
        for (int db = 0; db < DB; ++db) attend_again<T, D>(a, keys, values, qf, w0, p.end, t, db, ref, inv, p.result(a, i), redo);
    }
}

// The same for few queries: the waves of a block share 32 of them and take the
// tiles of 32 keys in turn, each with stages of its own in LDS (no barrier
// between tiles), and are joined at the end.
template <typename T, int D>
__global__ __launch_bounds__((64 * WaveLds<T, D>::kWaves), 1) void attn_fwd_shared_kernel(const AttnIn<T> a) {
    constexpr int NS = D / 16, NW = WaveLds<T, D>::kWaves, kStage = WaveLds<T, D>::kStage;
    typedef Tile<T, D, 32> Tl;
    extern __shared__ __align__(16) unsigned char lds[];
    float2 *stats = reinterpret_cast<float2 *>(lds + WaveLds<T, D>::kBytes);  // reference and 1 / sum of each query
    uint32_t &again = *reinterpret_cast<uint32_t *>(stats + 32);              // queries to form again

    const Place<T, D> p(a, 32);
    const int lane = threadIdx.x & 63, col = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int i = p.q0 + col, t = p.first + i, columns = min(32, a.L - p.q0);
    if (p.q0 >= p.len) {
        for (int e = threadIdx.x; e < columns * D; e += 64 * NW) narrow(p.result(a, p.q0 + e / D) + e % D, 0.f);
        if (a.lse != nullptr && (int)threadIdx.x < columns) *p.sums(a, p.q0 + threadIdx.x) = 0.f;
        return;
    }
    Frag<T> qf[NS];
#pragma unroll
    for (int s = 0; s < NS; ++s) load_frag(qf[s], p.query(a, i) + 16 * s + 8 * h, i < p.len);
    const int t0 = p.first + p.q0, t1 = min(t0 + 32, p.end) - 1;
    const Walk<32> walk(t0, t1, p.first, a.window, a.sinks);
    const Keys<T, D> keys = p.keys(a), values = p.values(a);
    unsigned char *own = lds + wave * 2 * kStage;
    Copier<Tl, 1> kcopy, vcopy;
    kcopy.init(a.ks.row * (int64_t)sizeof(T), 0, lane);
    vcopy.init(a.vs.row * (int64_t)sizeof(T), 0, lane);
    const auto stage = [&](int n, unsigned char *kl) {
        const int j0 = walk.start(n);
        if (j0 >= p.first) {
            const int rows = min((n < walk.nsink ? walk.sunk : p.end) - j0, 32);
            kcopy.copy(lds_addr(kl), keys.of(j0), rows);
            vcopy.copy(lds_addr(kl + Tl::kBytes), values.of(j0), rows);
        } else {
            Tl::template gather<64>(kl, [&](int r) { return walk.held(n, j0 + r, a.sinks, p.end) ? keys.of(j0 + r) : nullptr; });
            Tl::template gather<64>(kl + Tl::kBytes, [&](int r) { return walk.held(n, j0 + r, a.sinks, p.end) ? values.of(j0 + r) : nullptr; });
        }
    };
    if (wave < walk.ntiles) stage(wave, own);
#pragma unroll
    for (int s = 0; s < NS; ++s) arrived(qf[s]);
    Running<T, D> run;
    run.init();
    int buf = 0;
    for (int n = wave; n < walk.ntiles; n += NW, buf ^= 1) {
        // the copies of this tile are the oldest; what was read of the other stage has arrived
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        if (n + NW < walk.ntiles) stage(n + NW, own + (buf ^ 1) * kStage);
        const unsigned char *kl = own + buf * kStage;
        const int j0 = walk.start(n);
        floatx16 s[1];
        scores<Tl>(kl, qf, lane, s);
        const bool whole = n < walk.nsink ? j0 + 32 <= walk.sunk
                                          : j0 >= 0 && j0 + 31 <= t0 && (t0 + 31 - j0 < a.window || j0 + 32 <= a.sinks);
        if (!whole) hide(s, walk, n, j0, t, t0, h, a.window, a.sinks);
        run.template take<Tl, 1>(s, a.c, kl + Tl::kBytes, lane);
    }
    if (threadIdx.x == 0) again = 0;  // (Join's barriers come before its use)
    Join<T, D, NW>::run(lds, run, wave, lane, columns, [&](int c, int d, float y, float m, float l) {
        const int ic = p.q0 + c;
        const bool live = ic < p.len;
        const float inv = 1.f / l;
        narrow(p.result(a, ic) + d, live ? y * inv : 0.f);
        if (d == 0) {
            stats[c] = float2{m == -kInf ? 0.f : m, inv};
            if (a.lse != nullptr) *p.sums(a, ic) = live ? (m + __builtin_amdgcn_logf(l)) * kLn2 : 0.f;
        }
        if (live && y - y != 0.f && l > 0.f && l < kInf) atomicOr(&again, 1u << c);
    });
    __syncthreads();
    // (a wave takes some of the elements)
    if (again != 0) {
        const bool redo = (again >> col & 1) != 0;
#pragma unroll 1
        for (int db = wave; db < D / 32; db += NW)
            attend_again<T, D>(a, keys, values, qf, t0, p.end, t, db, stats[col].x, stats[col].y, p.result(a, i), redo);
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
    const int64_t blocks = batch * in.heads * ((in.L + kQueries - 1) / kQueries);
    if (few_queries<T, D>(blocks, in.L, in.window, in.positions != nullptr)) {
        constexpr int kLds = WaveLds<T, D>::kBytes + 32 * (int)sizeof(float2) + 16;
        const hipError_t e = allow_lds<attn_fwd_shared_kernel<T, D>>(kLds);
        if (e != hipSuccess) return e;
        attn_fwd_shared_kernel<T, D><<<dim3((uint32_t)(batch * in.heads * ((in.L + 31) / 32))), dim3(64 * WaveLds<T, D>::kWaves), kLds, stream>>>(in);
        return hipGetLastError();
    }
    constexpr int kLds = 2 * 2 * Tile<T, D, sizeof(T) == 2 ? 64 : 32>::kBytes;
    const hipError_t e = allow_lds<attn_fwd_kernel<T, D>>(kLds);
    if (e != hipSuccess) return e;
    attn_fwd_kernel<T, D><<<dim3((uint32_t)blocks), dim3(256), kLds, stream>>>(in);
    return hipGetLastError();
}

template <typename T>
hipError_t attn_fwd_typed(const AttnArgs &a, hipStream_t stream) {
    const AttnIn<T> in{static_cast<const T *>(a.q), static_cast<const T *>(a.k), static_cast<const T *>(a.v),
                       static_cast<T *>(a.kc), static_cast<T *>(a.vc), a.positions, a.lengths, static_cast<T *>(a.y), a.lse,
                       a.qs, a.ks, a.vs, (int64_t)a.window + a.sinks, a.seqlen, a.heads, a.kvheads,
                       a.window, a.sinks, a.scale * kLog2e};
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
