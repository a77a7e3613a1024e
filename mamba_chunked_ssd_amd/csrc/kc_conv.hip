// kc_conv.hip -- the short causal convolution of a layer's x, B and C, one
// filter of 2..4 taps per channel: forward over prompts, backward, one token.
//
//   p_t = bias + sum_k w_k x_{t-W+1+k} ,  y_t = act(p_t)
//
// Bound by memory: each element of x is read and each of y written once,
// against 2 W + about 10 vector operations.  A lane owns the channels of one
// load and walks a run of tokens with the last W - 1 inputs in registers, so
// only the run's first W - 1 rows are read twice (from the L2).  The lanes of a
// wave take consecutive channels, so every access is one contiguous piece of a
// row, and rows come and go through raw buffers over a group of tokens, so
// that the ends of sequences and rows need no branch.
#include <algorithm>

#include "ssd_launch.h"
#include "ssd_ops_device.h"
#include "ssd_ops_internal.h"

namespace ssd {
namespace {

template <typename T>
struct ConvIn {
    const T *x, *init;
    const float *weight, *bias;
    const int32_t *lengths;
    int64_t xb, xr;  // strides of x
    int L, C, nvec, nvb;
    bool silu;
};

__device__ __forceinline__ int conv_length(const int32_t *lengths, int b, int L) {
    return lengths == nullptr ? L : min(max(lengths[b], 0), L);
}

template <int W, int V>
__device__ __forceinline__ void load_filter(const float *weight, const float *bias, int c0, float (&w)[W][V],
                                            float (&bs)[V]) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
#pragma unroll
        for (int k = 0; k < W; ++k) w[k][e] = weight[(int64_t)(c0 + e) * W + k];
        bs[e] = bias != nullptr ? bias[c0 + e] : 0.f;
    }
}

// Input row t of a sequence: the initial state's rows stand before row 0.
template <typename T, int W, int V>
__device__ __forceinline__ Raw<T, V> conv_row(const ConvIn<T> &a, int b, int t, int len, int c0) {
    Raw<T, V> r;
    r.zero();
    if (t < 0) {
        if (a.init != nullptr) r.load(a.init + ((int64_t)b * (W - 1) + (W - 1) + t) * a.C + c0);
    } else if (t < len) {
        r.load(a.x + b * a.xb + t * a.xr + c0);
    }
    return r;
}

// Rows first .. of a group of U tokens, none behind `rows`.
template <int U, typename T>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t group_rows(const T *first, int64_t row, int rows) {
    return uniform_rsrc(first, (uint32_t)min(max(rows, 0), U) * (uint32_t)(row * (int64_t)sizeof(T)));
}

// A wave takes a run of 16 tokens, eight at a time with the next eight's loads
// in flight.  Longer runs read the filters less often, from the L2, and were
// slower (4 x 4096 tokens of 5376 channels, fp32: 130 us with 16, 137 with 32,
// 149 with 128).  8 x 4096 tokens of 5376 channels, bf16: 134 us, 5.25 TB/s,
// 98 % of a copy's rate.
constexpr int kFwdRun = 16;
template <typename Tin, typename Tout, int W, int V>
__global__ __launch_bounds__(256) void kc_conv_fwd(ConvIn<Tin> a, Tout *__restrict__ y, Tin *final_state, int nruns) {
    constexpr int U = 8;
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int vec = (int)(blockIdx.x % a.nvb) * 64 + lane, rn = (int)(blockIdx.x / a.nvb) * 4 + wave;
    if (rn >= nruns) return;
    const bool mine = vec < a.nvec;
    const int b = blockIdx.y, c0 = mine ? vec * V : 0;
    const int t0 = rn * kFwdRun, t1 = min(t0 + kFwdRun, a.L);
    const int len = conv_length(a.lengths, b, a.L), tend = min(t1, len);
    const uint32_t xoff = mine ? c0 * (uint32_t)sizeof(Tin) : kNowhere, xrow = (uint32_t)(a.xr * (int64_t)sizeof(Tin));
    const uint32_t yoff = mine ? c0 * (uint32_t)sizeof(Tout) : kNowhere, yrow = (uint32_t)a.C * (uint32_t)sizeof(Tout);
    const Tin *xp = a.x + b * a.xb + t0 * a.xr;
    Tout *yp = y + ((int64_t)b * a.L + t0) * a.C;

    Raw<Tin, V> in[U], next[U];
    auto fetch = [&](int t, Raw<Tin, V>(&to)[U]) {
        const __amdgpu_buffer_rsrc_t r = group_rows<U>(xp, a.xr, tend - t);
#pragma unroll
        for (int u = 0; u < U; ++u) to[u].load(r, xoff + u * xrow);
        xp += U * a.xr;
    };
    fetch(t0, in);
    float w[W][V], bs[V], win[W][V];  // win[k]: x_{t - W + 1 + k}
    load_filter<W, V>(a.weight, a.bias, c0, w, bs);
#pragma unroll
    for (int k = 1; k < W; ++k) conv_row<Tin, W, V>(a, b, t0 - W + k, len, c0).unpack(win[k]);

    // The first run's lanes hold the initial state already when they write the
    // final one, so the two may be the same buffer.
    if (rn == 0 && final_state != nullptr && mine) {
        Raw<Tin, V> keep[W - 1];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) keep[k] = conv_row<Tin, W, V>(a, b, len - (W - 1) + k, len, c0);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            float f[V];
            keep[k].unpack(f);
            store_n<V>(final_state + ((int64_t)b * (W - 1) + k) * a.C + c0, f);  // exact: the values are Tin's
        }
    }

    for (int t = t0; t < t1; t += U) {
        fetch(t + U, next);
        const __amdgpu_buffer_rsrc_t ry = group_rows<U>(yp, a.C, t1 - t);
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int k = 0; k < W - 1; ++k)
#pragma unroll
                for (int e = 0; e < V; ++e) win[k][e] = win[k + 1][e];
            in[u].unpack(win[W - 1]);
            float out[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float p = bs[e];
#pragma unroll
                for (int k = 0; k < W; ++k) p = fmaf(w[k][e], win[k][e], p);
                if (a.silu) p *= logistic(p);
                out[e] = t + u < len ? p : 0.f;
            }
            store_n<V>((const Tout *)nullptr, ry, yoff + u * yrow, out);
            in[u] = next[u];
        }
        yp += U * (int64_t)a.C;
    }
}

// Backward: with d_t = dy_t act'(p_t) (0 behind the end),
//   dx_s = sum_k w_k d_{s+W-1-k} ,  dw_k = sum_t d_t x_{t-W+1+k} ,  db = sum_t d_t .
// A wave walks t over its strip, four tokens at a time with the next four's
// loads in flight, and over one group beyond it, whose d_t it forms again:
// dx_{t-W+1} is complete at t.  Rows come and go through raw buffers over the
// group; what a sequence's end changes is a path of its own.  dw and db stay in registers over the
// strip, are joined over the block's four strips in LDS and leave one row of
// partial sums per block, which kc_conv_sums adds in a fixed order.  They are
// held in 64 bits, where a product of two fp32 numbers is exact, and rounded to
// fp32 three times, as a strip's, a block's and the whole sum, however time is
// cut.  Bound by memory: 2 x 2048 tokens of 5376 channels, bf16 with dy in fp32,
// 38 us of which the 176 MB that must move take 34 at a copy's rate (sums 4 us
// more); 4 x 4096 tokens fp32 228 us, its bytes 204.  The 64 bits cost 5 % of
// the first, whose registers then leave two waves a SIMD, and 1 % of the second.
// Measured and not kept: partial sums as two floats (47 us for both kernels
// against 46), 64-bit sums in LDS, added to every four tokens (44, but 231 fp32).
// Registers for three waves a SIMD are asked for where x, dy and dx are all bf16
// (4 x 4096 tokens: 125 us, 132 with the two that the compiler leaves by itself);
// with any of them in fp32 they spill (the first case 50 us against 45).
constexpr int kGroup = 4;  // tokens; at least W - 1

template <typename Tin, typename Tdy, typename Tdx, int W, int V>
__global__ __launch_bounds__(256, sizeof(Tin) + sizeof(Tdy) + sizeof(Tdx) == 6 ? 3 : 1)
void kc_conv_bwd(ConvIn<Tin> a, const Tdy *__restrict__ dy, int64_t dyb, int64_t dyr, const float *__restrict__ dfinal,
                 Tdx *__restrict__ dx, float *__restrict__ dinit, float *__restrict__ partials, int strip, int nstrips) {
    constexpr int U = kGroup, R = (W + 1) * V;
    __shared__ float red[4 * R * 64];
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int vb = blockIdx.x % a.nvb, sb = blockIdx.x / a.nvb;
    const int vec = vb * 64 + lane, st = sb * 4 + wave, b = blockIdx.y, c0 = vec * V;
    const bool mine = vec < a.nvec;
    const int len = conv_length(a.lengths, b, a.L);

    double dw[W][V], db[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        db[e] = 0.0;
#pragma unroll
        for (int k = 0; k < W; ++k) dw[k][e] = 0.0;
    }
    if (st < nstrips) {
        const int t0 = st * strip, t1 = min(t0 + strip, a.L), tend = min(t1 + W - 1, len);
        const uint32_t xoff = mine ? c0 * (uint32_t)sizeof(Tin) : kNowhere;
        const uint32_t yoff = mine ? c0 * (uint32_t)sizeof(Tdy) : kNowhere;
        const uint32_t goff = mine ? c0 * (uint32_t)sizeof(Tdx) : kNowhere;
        const uint32_t xrow = (uint32_t)(a.xr * (int64_t)sizeof(Tin)), yrow = (uint32_t)(dyr * (int64_t)sizeof(Tdy));
        const uint32_t grow = (uint32_t)a.C * (uint32_t)sizeof(Tdx);
        const Tin *xp = a.x + b * a.xb + t0 * a.xr;
        const Tdy *yp = dy + b * dyb + t0 * dyr;
        Tdx *gp = dx + ((int64_t)b * a.L + t0 - (W - 1)) * a.C;

        float w[W][V], bs[V], win[W][V], dp[W][V];  // dp[k]: d_{t - W + 1 + k}
        load_filter<W, V>(a.weight, a.bias, mine ? c0 : 0, w, bs);
#pragma unroll
        for (int k = 0; k < W; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e) dp[k][e] = 0.f;
#pragma unroll
        for (int k = 1; k < W; ++k) conv_row<Tin, W, V>(a, b, t0 - W + k, len, mine ? c0 : 0).unpack(win[k]);

        Raw<Tin, V> in[U];
        Raw<Tdy, V> up[U];
        auto fetch = [&](int t) {
            const __amdgpu_buffer_rsrc_t rx = group_rows<U>(xp, a.xr, tend - t), ry = group_rows<U>(yp, dyr, tend - t);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                in[u].load(rx, xoff + u * xrow);
                up[u].load(ry, yoff + u * yrow);
            }
            xp += U * a.xr;
            yp += U * dyr;
        };
        const int live = min(t1, len);  // the strip's own tokens end here
        // ENDS: a group that reaches behind them.  Rows behind a sequence's end get 0 by selection and add nothing: the
        // windows of the first still hold the last inputs, and 0 times one that is not finite would be NaN.
        auto group = [&](int t, auto ENDS) {
            constexpr bool ends = decltype(ENDS)::value;
            float x[U][V], d[U][V], g[U][V];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                in[u].unpack(x[u]);
                up[u].unpack(d[u]);
            }
            fetch(t + U);
#pragma unroll
            for (int u = 0; u < U; ++u) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
#pragma unroll
                    for (int k = 0; k < W - 1; ++k) {
                        win[k][e] = win[k + 1][e];
                        dp[k][e] = dp[k + 1][e];
                    }
                    win[W - 1][e] = x[u][e];
                    float de = d[u][e];
                    if (a.silu) {
                        float p = bs[e];
#pragma unroll
                        for (int k = 0; k < W; ++k) p = fmaf(w[k][e], win[k][e], p);
                        const float sg = logistic(p);
                        // silu'(p) = s (1 + p (1 - s))
                        de *= sg * fmaf(p, 1.f - sg, 1.f);
                        if constexpr (ends) de = t + u < len ? de : 0.f;
                    }
                    dp[W - 1][e] = de;
                    if (!ends || t + u < live) {
                        db[e] += de;
#pragma unroll
                        for (int k = 0; k < W; ++k) dw[k][e] = fma((double)de, (double)win[k][e], dw[k][e]);
                    }
                    g[u][e] = 0.f;
#pragma unroll
                    for (int k = 0; k < W; ++k) g[u][e] = fmaf(w[k][e], dp[W - 1 - k][e], g[u][e]);
                }
            }
            const int s0 = t - (W - 1);  // the row of g[0]
            if (ends && dfinal != nullptr && s0 + U > len - (W - 1) && s0 < len && mine) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int i = s0 + u - len + (W - 1);  // its row in the final state
                    if (i >= 0 && i < W - 1) {
                        Raw<float, V> r;
                        float f[V];
                        r.load(dfinal + ((int64_t)b * (W - 1) + i) * a.C + c0);
                        r.unpack(f);
#pragma unroll
                        for (int e = 0; e < V; ++e) g[u][e] += f[e];
                    }
                }
            }
            if (ends && s0 + U > len) {  // whatever the filter
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int e = 0; e < V; ++e) g[u][e] = s0 + u < len ? g[u][e] : 0.f;
            }
            // the strip's first rows have no place here: they end the strip before, or the initial state
            const bool first = t == t0;
            if (first && st == 0 && dinit != nullptr && mine) {
#pragma unroll
                for (int u = 0; u < W - 1; ++u) store_n<V>(dinit + ((int64_t)b * (W - 1) + u) * a.C + c0, g[u]);
            }
            const __amdgpu_buffer_rsrc_t rg = group_rows<U>(gp, a.C, t1 - s0);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (u >= W - 1 || !first) store_n<V>((const Tdx *)nullptr, rg, goff + u * grow, g[u]);
            gp += U * (int64_t)a.C;
        };
        fetch(t0);
        int t = t0;
        for (; t + U <= live; t += U) group(t, std::false_type{});
        for (; t < t1 + U; t += U) group(t, std::true_type{});
    }

#pragma unroll
    for (int e = 0; e < V; ++e) {
#pragma unroll
        for (int k = 0; k < W; ++k) red[(wave * R + k * V + e) * 64 + lane] = (float)dw[k][e];
        red[(wave * R + W * V + e) * 64 + lane] = (float)db[e];
    }
    __syncthreads();
    const int nsb = (nstrips + 3) / 4;
    float *out = partials + ((int64_t)b * nsb + sb) * (W + 1) * a.C;
    for (int i = threadIdx.x; i < R * 64; i += 256) {
        // consecutive threads take consecutive channels of one tap
        const int k = i / (V * 64), cl = i % (V * 64), c = vb * 64 * V + cl;
        double sum = 0.0;
#pragma unroll
        for (int q = 0; q < 4; ++q) sum += red[(q * R + k * V + cl % V) * 64 + cl / V];
        if (c < a.C) out[(int64_t)k * a.C + c] = (float)sum;
    }
}

// dweight and dbias: column (tap, channel) summed over the rows of partial
// sums in a fixed order and 64 bits, sixteen threads a column, each every
// sixteenth row: few channels over long inputs leave hundreds of rows to few
// columns.
__global__ __launch_bounds__(256) void kc_conv_sums(const float *__restrict__ partials, int64_t parts, int C, int W,
                                                    float *__restrict__ dweight, float *__restrict__ dbias) {
    constexpr int COLS = 16, SLICES = 16;
    __shared__ double part[256];
    const int64_t cols = (int64_t)(W + 1) * C, col = (int64_t)blockIdx.x * COLS + threadIdx.x % COLS;
    const int q = threadIdx.x / COLS;
    double sum = 0.0;
    if (col < cols) {
#pragma unroll 4
        for (int64_t p = q; p < parts; p += SLICES) sum += (double)partials[p * cols + col];
    }
    part[threadIdx.x] = sum;
    __syncthreads();
    if (q == 0 && col < cols) {
#pragma unroll
        for (int k = 1; k < SLICES; ++k) sum += part[k * COLS + threadIdx.x];
        const int k = (int)(col / C), c = (int)(col % C);
        if (k < W) dweight[(int64_t)c * W + k] = (float)sum;
        else if (dbias != nullptr) dbias[c] = (float)sum;
    }
}

// One token per sequence: all W - 1 kept rows and x in, y and the shifted rows out.
template <typename Tin, typename Tout, int W, int V>
__global__ __launch_bounds__(256) void kc_conv_step(ConvIn<Tin> a, Tin *state, Tout *__restrict__ y) {
    const int64_t gid = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int b = blockIdx.y;
    if (gid >= a.nvec) return;
    const int c0 = (int)gid * V;
    Raw<Tin, V> row[W];
    Tin *sp = state + (int64_t)b * (W - 1) * a.C + c0;
    row[W - 1].load(a.x + b * a.xb + c0);
#pragma unroll
    for (int k = 0; k < W - 1; ++k) row[k].load(sp + (int64_t)k * a.C);
    float w[W][V], p[V], f[V];
    load_filter<W, V>(a.weight, a.bias, c0, w, p);
#pragma unroll
    for (int k = 0; k < W; ++k) {
        row[k].unpack(f);
        if (k > 0) store_n<V>(sp + (int64_t)(k - 1) * a.C, f);
#pragma unroll
        for (int e = 0; e < V; ++e) p[e] = fmaf(w[k][e], f[e], p[e]);
    }
    if (a.silu) {
#pragma unroll
        for (int e = 0; e < V; ++e) p[e] *= logistic(p[e]);
    }
    store_n<V>(y + (int64_t)b * a.C + c0, p);
}

// Whether V-element loads and stores fit: whole vectors in a row, every row
// and buffer aligned to them.
template <typename T>
bool vec_ok(const void *p, int V) {
    return (uintptr_t)p % (V * sizeof(T)) == 0;
}

template <typename Tin>
ConvIn<Tin> conv_in(const ConvArgs &a, int V, int bx) {
    ConvIn<Tin> in;
    in.x = static_cast<const Tin *>(a.x);
    in.init = static_cast<const Tin *>(a.init);
    in.weight = a.weight;
    in.bias = a.bias;
    in.lengths = a.lengths;
    in.xb = a.xs.batch;
    in.xr = a.xs.row;
    in.L = a.seqlen;
    in.C = a.channels;
    in.nvec = a.channels / V;
    in.nvb = (in.nvec + bx - 1) / bx;
    in.silu = a.silu;
    return in;
}

// Whether four channels a lane leave at most one lane in four of their waves idle.
bool waves_full(int channels) { return 4 * (int64_t)channels >= 3 * ((channels + 255) / 256 * (int64_t)256); }

template <typename Tin, typename Tout, int W, int V>
hipError_t fwd(const ConvArgs &a, hipStream_t stream) {
    const ConvIn<Tin> in = conv_in<Tin>(a, V, 64);
    const int nruns = a.seqlen > 0 ? (a.seqlen + kFwdRun - 1) / kFwdRun : 1;
    const int64_t blocks = (int64_t)in.nvb * ((nruns + 3) / 4);
    return launch_kernel(kc_conv_fwd<Tin, Tout, W, V>, dim3((unsigned)blocks, (unsigned)a.batch), dim3(256), 0, stream,
                         LaunchEvents{}, in, static_cast<Tout *>(a.y), static_cast<Tin *>(a.final_state), nruns);
}

template <typename Tin, typename Tdy, typename Tdx, int W, int V>
hipError_t bwd(const ConvArgs &a, const ConvBwdPlan &plan, hipStream_t stream) {
    const ConvIn<Tin> in = conv_in<Tin>(a, V, 64);
    if (a.batch > 0) {
        const int64_t blocks = (int64_t)in.nvb * ((plan.nstrips + 3) / 4);
        const hipError_t e = launch_kernel(
            kc_conv_bwd<Tin, Tdy, Tdx, W, V>, dim3((unsigned)blocks, (unsigned)a.batch), dim3(256), 0, stream,
            LaunchEvents{}, in, static_cast<const Tdy *>(a.dy), a.dys.batch, a.dys.row, a.dfinal,
            static_cast<Tdx *>(a.dx), a.dinit, a.partials, plan.strip, plan.nstrips);
        if (e != hipSuccess) return e;
    }
    const int64_t cols = (int64_t)(W + 1) * a.channels;
    return launch_kernel(kc_conv_sums, dim3((unsigned)((cols + 15) / 16)), dim3(256), 0, stream, LaunchEvents{},
                         (const float *)a.partials, plan.parts, a.channels, W, a.dweight, a.dbias);
}

template <typename Tin, typename Tout, int W, int V>
hipError_t step(const ConvArgs &a, hipStream_t stream) {
    const ConvIn<Tin> in = conv_in<Tin>(a, V, 256);
    return launch_kernel(kc_conv_step<Tin, Tout, W, V>, dim3((unsigned)in.nvb, (unsigned)a.batch), dim3(256), 0, stream,
                         LaunchEvents{}, in, static_cast<Tin *>(const_cast<void *>(a.init)), static_cast<Tout *>(a.y));
}

// Four channels a lane where every operand's rows are whole pieces of four and
// the waves they fill are nearly full, else one.  Measured (4 x 4096 tokens of
// 5376 channels): forward fp32 136 us with four, 148 with one, bf16 78 and 84,
// backward fp32 227 and 234.  264 channels, which fill half of two waves of
// fours: fp32 8 x 4096 tokens 22.1 us with four, 19.9 with one, and backward
// 35.6 and 33.0.
template <typename Tin, typename Tout, int W>
hipError_t fwd_v(const ConvArgs &a, hipStream_t s) {
    const bool v = a.channels % 4 == 0 && a.xs.batch % 4 == 0 && a.xs.row % 4 == 0 && vec_ok<Tin>(a.x, 4) &&
                   vec_ok<Tin>(a.init, 4) && vec_ok<Tout>(a.y, 4) && vec_ok<Tin>(a.final_state, 4);
    return v && waves_full(a.channels) ? fwd<Tin, Tout, W, 4>(a, s) : fwd<Tin, Tout, W, 1>(a, s);
}
template <int W>
hipError_t fwd_w(const ConvArgs &a, hipStream_t s) {
    if (!a.in_bf16) return fwd_v<float, float, W>(a, s);
    return a.y_bf16 ? fwd_v<uint16_t, uint16_t, W>(a, s) : fwd_v<uint16_t, float, W>(a, s);
}

template <typename Tin, typename Tdy, typename Tdx, int W>
hipError_t bwd_v(const ConvArgs &a, const ConvBwdPlan &p, hipStream_t s) {
    const bool v = a.channels % 4 == 0 && a.xs.batch % 4 == 0 && a.xs.row % 4 == 0 && a.dys.batch % 4 == 0 &&
                   a.dys.row % 4 == 0 && vec_ok<Tin>(a.x, 4) && vec_ok<Tin>(a.init, 4) && vec_ok<Tdy>(a.dy, 4) &&
                   vec_ok<Tdx>(a.dx, 4) && vec_ok<float>(a.dfinal, 4) && vec_ok<float>(a.dinit, 4);
    return v && waves_full(a.channels) ? bwd<Tin, Tdy, Tdx, W, 4>(a, p, s) : bwd<Tin, Tdy, Tdx, W, 1>(a, p, s);
}

template <int W>
hipError_t bwd_w(const ConvArgs &a, const ConvBwdPlan &p, hipStream_t s) {
    if (!a.in_bf16) return bwd_v<float, float, float, W>(a, p, s);
    if (a.y_bf16)
        return a.dx_bf16 ? bwd_v<uint16_t, uint16_t, uint16_t, W>(a, p, s)
                         : bwd_v<uint16_t, uint16_t, float, W>(a, p, s);
    return a.dx_bf16 ? bwd_v<uint16_t, float, uint16_t, W>(a, p, s) : bwd_v<uint16_t, float, float, W>(a, p, s);
}

template <int W>
hipError_t step_w(const ConvArgs &a, hipStream_t s) {
    if (!a.in_bf16) {
        const bool v = a.channels % 4 == 0 && a.xs.batch % 4 == 0 && vec_ok<float>(a.x, 4) &&
                       vec_ok<float>(a.init, 4) && vec_ok<float>(a.y, 4);
        return v ? step<float, float, W, 4>(a, s) : step<float, float, W, 1>(a, s);
    }
    const bool v = a.channels % 4 == 0 && a.xs.batch % 4 == 0 && vec_ok<uint16_t>(a.x, 4) &&
                   vec_ok<uint16_t>(a.init, 4) && (uintptr_t)a.y % 16 == 0;
    if (a.y_bf16) return v ? step<uint16_t, uint16_t, W, 4>(a, s) : step<uint16_t, uint16_t, W, 1>(a, s);
    return v ? step<uint16_t, float, W, 4>(a, s) : step<uint16_t, float, W, 1>(a, s);
}

}  // namespace

hipError_t launch_conv_fwd(const ConvArgs &a, hipStream_t stream) {
    switch (a.width) {
        case 2: return fwd_w<2>(a, stream);
        case 3: return fwd_w<3>(a, stream);
        case 4: return fwd_w<4>(a, stream);
        default: return hipErrorInvalidValue;
    }
}

hipError_t launch_conv_bwd(const ConvArgs &a, const ConvBwdPlan &plan, hipStream_t stream) {
    switch (a.width) {
        case 2: return bwd_w<2>(a, plan, stream);
        case 3: return bwd_w<3>(a, plan, stream);
        case 4: return bwd_w<4>(a, plan, stream);
        default: return hipErrorInvalidValue;
    }
}

hipError_t launch_conv_step(const ConvArgs &a, hipStream_t stream) {
    switch (a.width) {
        case 2: return step_w<2>(a, stream);
        case 3: return step_w<3>(a, stream);
        case 4: return step_w<4>(a, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace ssd
