// kn_norm_bwd.hip -- gradients through the RMS norm.
//
//   du = r w dy - u r^3 mean(w dy u) + d_residual ,  dw = sum_rows dy u r
//
// formed as du = r (w dy - z g) + d_residual with z = u r and g = r mean(w dy u):
// z is of order 1 and g of the order of w dy whatever u's size, where r^3 leaves
// fp32's range from |u| of 1e13 up and, with eps 0, of 1e-13 down.
//
// Bound by memory, laid out as the forward pass: a row stays in the registers
// of a wave (a block) between its two sums, taken in one pass, and du.  The
// columns' sums of dy u r stay in the lanes that own the columns over the rows
// that a wave takes; what blocks leave is added in a fixed order, in 64 bits, by
// a second kernel.
//
// Measured: 2 x 2048 tokens of 2560 channels, bf16 with an fp32 stream 36 us and
// 4.4 for the sums (16 threads a column, a load at a time: 11), 4.1 TB/s together;
// 3 x 1021 tokens of 264 fp32 channels 6.5 and 4.2.
#include <algorithm>

#include "kn_norm.h"

namespace ssd {
namespace {

struct NormBwdIn {
    const void *dy, *u, *dres;
    const float *weight;
    const int32_t *lengths;
    void *dx, *dresidual;
    float *partials;  // (gridDim.x, C), or null
    Strides dys, us, drs;
    uint32_t rows;
    int L, C;
    float eps;
    Stored x, res;
};

// One row's r and g, from its sums.
struct Factors {
    float r, g;
};
__device__ __forceinline__ Factors factors(float uu, float wdu, int C, float eps) {
    const float r = rsqrtf(uu / (float)C + eps);
    return Factors{r, r * (wdu / (float)C)};
}
template <int TPR>
__device__ __forceinline__ void row_sums(float &p, float &q, float2 *room) {
    p = lane_total<16>(p);
    q = lane_total<16>(q);
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(p), __float_as_uint(q), false, false);
    // rows 0 and 2 of a wave now hold p's parts, rows 1 and 3 q's
    float s = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(s), __float_as_uint(s), false, false);
    s = __uint_as_float(b[0]) + __uint_as_float(b[1]);
    const auto c = __builtin_amdgcn_permlane16_swap(__float_as_uint(s), __float_as_uint(s), false, false);
    p = __uint_as_float(c[0]);
    q = __uint_as_float(c[1]);
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) room[threadIdx.x >> 6] = float2{p, q};
        __syncthreads();
        p = (room[0].x + room[1].x) + (room[2].x + room[3].x);
        q = (room[0].y + room[1].y) + (room[2].y + room[3].y);
    }
}

// A lane keeps its columns' sums of dy u r over the rows that its wave (block)
// takes, 256 at most before they are added to the block's row of partial sums.
template <typename TY, typename TU, int TPR, int NV>
__global__ __launch_bounds__(256) void norm_bwd_kernel(const NormBwdIn a) {
    __shared__ float2 room[2][4];
    extern __shared__ float sums[];  // a wave to a row: (3, C rounded up to 8)
    const int lane = threadIdx.x % TPR, C = a.C;
    uint32_t row = blockIdx.x, step = gridDim.x;
    if constexpr (TPR == 64) {
        row = row * 4 + (uint32_t)__builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
        step *= 4;
    }
    float dw[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[i][e] = 0.f;
    const auto at_piece = [&](int i) { return (i * TPR + lane) * 8; };
    int turn = 0;
    for (uint64_t at = row; at < a.rows; at += step) {
        const Place p = place_of((uint32_t)at, (uint32_t)a.L, a.lengths);
        const int64_t out = (int64_t)at * C;
        if (!p.live) {
            zero_row<TPR>(a.x, a.dx, out, C);
            if (a.dresidual != nullptr) zero_row<TPR>(a.res, a.dresidual, out, C);
            continue;
        }
        Eight<TU> u[NV], dres[NV];
        Eight<TY> dy[NV];
        Eight<float> wt[NV];
        const TU *ur = static_cast<const TU *>(a.u) + p.b * a.us.batch + p.t * a.us.row;
        const TU *dr = static_cast<const TU *>(a.dres) + p.b * a.drs.batch + p.t * a.drs.row;
        const TY *yr = static_cast<const TY *>(a.dy) + p.b * a.dys.batch + p.t * a.dys.row;
        for_pieces<NV>([&](auto i, auto last) {
            load_piece<last>(u[i], ur, at_piece(i), C);
            load_piece<last>(dy[i], yr, at_piece(i), C);
        });
        if (a.weight != nullptr)
            for_pieces<NV>([&](auto i, auto last) { load_piece<last>(wt[i], a.weight, at_piece(i), C); });
        else
            for_pieces<NV>([&](auto i, auto) { wt[i].v[0] = wt[i].v[1] = floatx4{1.f, 1.f, 1.f, 1.f}; });
        if (a.dres != nullptr)
            for_pieces<NV>([&](auto i, auto last) { load_piece<last>(dres[i], dr, at_piece(i), C); });
        else
            for_pieces<NV>([&](auto i, auto) { dres[i].zero(); });
        float uu = 0.f, wdu = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float x = u[i].get(e);
                uu = fmaf(x, x, uu);
                wdu = fmaf(wt[i].get(e) * dy[i].get(e), x, wdu);
            }
        row_sums<TPR>(uu, wdu, room[turn]);
        turn ^= 1;
        const Factors f = factors(uu, wdu, C, a.eps);
        for_pieces<NV>([&](auto i, auto last) {
            float du[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float z = u[i].get(e) * f.r, g = dy[i].get(e);
                dw[i][e] = fmaf(g, z, dw[i][e]);
                du[e] = fmaf(f.r, fmaf(-z, f.g, wt[i].get(e) * g), dres[i].get(e));
            }
            store_as<last>(a.x, a.dx, out, at_piece(i), C, du);
            if (a.dresidual != nullptr) store_as<last>(a.res, a.dresidual, out, at_piece(i), C, du);
        });
    }
    if (a.partials == nullptr) return;
    if constexpr (TPR == 64) {
        // waves 1 .. 3 hand theirs to wave 0, in that order
        const int wide = (C + 7) / 8 * 8, wave = threadIdx.x >> 6;
        if (wave > 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c0 = (i * TPR + lane) * 8;
                if (c0 < C) __builtin_memcpy(sums + (wave - 1) * wide + c0, dw[i], 32);
            }
        }
        __syncthreads();
        if (wave > 0) return;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c0 = (i * TPR + lane) * 8;
            if (c0 < C) {
#pragma unroll
                for (int v = 0; v < 3; ++v)
#pragma unroll
                    for (int e = 0; e < 8; ++e) dw[i][e] += sums[v * wide + c0 + e];
            }
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c0 = (i * TPR + lane) * 8;
        store_piece<true>(a.partials + (int64_t)blockIdx.x * C, c0, C, dw[i]);
    }
}

// Rows of any length: twice over the row, the sums of dy u r added to the
// block's row of partial sums (a thread's own columns) row by row.
template <typename TY, typename TU>
__global__ __launch_bounds__(256) void norm_bwd_long_kernel(const NormBwdIn a) {
    __shared__ float2 room[2][4];
    const int C = a.C;
    float *own = a.partials + (int64_t)blockIdx.x * C;
    if (a.partials != nullptr)
        for (int c0 = threadIdx.x * 8; c0 < C; c0 += 2048)
            for (int c = c0; c < min(c0 + 8, C); ++c) own[c] = 0.f;
    int turn = 0;
    for (uint64_t at = blockIdx.x; at < a.rows; at += gridDim.x, turn ^= 1) {
        const Place p = place_of((uint32_t)at, (uint32_t)a.L, a.lengths);
        const int stop = p.live ? C : 0;
        const TU *ur = static_cast<const TU *>(a.u) + p.b * a.us.batch + p.t * a.us.row;
        const TU *dr = static_cast<const TU *>(a.dres) + p.b * a.drs.batch + p.t * a.drs.row;
        const TY *yr = static_cast<const TY *>(a.dy) + p.b * a.dys.batch + p.t * a.dys.row;
        double tu = 0.0, td = 0.0;
        Eight<TU> u, dres;
        Eight<TY> dy;
        Eight<float> v;
        for (int c0 = threadIdx.x * 8; c0 < stop; c0 += 2048) {
            load_piece<true>(u, ur, c0, stop);
            load_piece<true>(dy, yr, c0, stop);
            if (a.weight != nullptr) load_piece<true>(v, a.weight, c0, stop);
            float s = 0.f, d = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float x = u.get(e), w = a.weight != nullptr ? v.get(e) : 1.f;
                s = fmaf(x, x, s);
                d = fmaf(w * dy.get(e), x, d);
            }
            tu += s;
            td += d;
        }
        float uu = (float)tu, wdu = (float)td;
        row_sums<256>(uu, wdu, room[turn]);
        Factors f = factors(uu, wdu, C, a.eps);
        if (!p.live) f = Factors{0.f, 0.f};
        const int64_t out = (int64_t)at * C;
        for (int c0 = threadIdx.x * 8; c0 < C; c0 += 2048) {
            load_piece<true>(u, ur, c0, stop);
            load_piece<true>(dy, yr, c0, stop);
            load_piece<true>(dres, dr, c0, a.dres != nullptr ? stop : 0);
            if (a.weight != nullptr) load_piece<true>(v, a.weight, c0, stop);
            float du[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float z = u.get(e) * f.r, g = dy.get(e), w = a.weight != nullptr ? v.get(e) : 1.f;
                du[e] = fmaf(f.r, fmaf(-z, f.g, w * g), dres.get(e));
                if (a.partials != nullptr && c0 + e < stop) own[c0 + e] = fmaf(g, z, own[c0 + e]);
            }
            store_as<true>(a.x, a.dx, out, c0, C, du);
            if (a.dresidual != nullptr) store_as<true>(a.res, a.dresidual, out, c0, C, du);
        }
    }
}

// dweight: the blocks' partial sums, a wave's width of columns by 16 slices of
// the blocks, in 64 bits.  Loads of several blocks are on their way at a time.
__global__ __launch_bounds__(1024) void norm_dweight_kernel(const float *partials, int parts, int C, float *dweight) {
    __shared__ double room[16][64];
    const int col = threadIdx.x & 63, slice = threadIdx.x >> 6;
    for (int base = blockIdx.x * 64; base < C; base += gridDim.x * 64) {
        const int c = base + col;
        double s = 0.0;
        if (c < C) {
            int p = slice;
            for (; p + 16 * 7 < parts; p += 16 * 8) {
                float v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = partials[(int64_t)(p + 16 * k) * C + c];
#pragma unroll
                for (int k = 0; k < 8; ++k) s += (double)v[k];
            }
            for (; p < parts; p += 16) s += (double)partials[(int64_t)p * C + c];
        }
        room[slice][col] = s;
        __syncthreads();
        if (slice == 0 && c < C) {
#pragma unroll
            for (int k = 1; k < 16; ++k) s += room[k][col];
            dweight[c] = (float)s;
        }
        __syncthreads();
    }
}

template <typename TY, typename TU>
hipError_t norm_bwd_typed(const NormBwdIn &a, int parts, hipStream_t stream) {
    const dim3 grid(parts), block(256);
    if (a.C > kNormBlockRow) {
        norm_bwd_long_kernel<TY, TU><<<grid, block, 0, stream>>>(a);
    } else if (a.C > kNormWaveRow) {
        with_pieces<3, 8>((a.C + 2047) / 2048, [&](auto n) { norm_bwd_kernel<TY, TU, 256, n><<<grid, block, 0, stream>>>(a); });
    } else {
        const size_t lds = a.partials != nullptr ? (size_t)3 * ((a.C + 7) / 8 * 8) * sizeof(float) : 0;
        with_pieces<1, 8>((a.C + 511) / 512, [&](auto n) { norm_bwd_kernel<TY, TU, 64, n><<<grid, block, lds, stream>>>(a); });
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_bwd(const NormArgs &a, const NormBwdPlan &plan, hipStream_t stream) {
    NormBwdIn in{a.in, a.residual, a.dres, a.weight, a.lengths, a.out, a.residual_out,
                 a.dweight != nullptr ? a.partials : nullptr, a.dys, a.rs, a.drs, (uint32_t)(a.batch * a.seqlen),
                 std::max(a.seqlen, 1), a.channels, a.eps, a.x, a.res};
    const bool y16 = a.y == Stored::bf16, u16 = a.res == Stored::bf16;
    hipError_t e;
    if (y16) e = u16 ? norm_bwd_typed<uint16_t, uint16_t>(in, plan.parts, stream) : norm_bwd_typed<uint16_t, float>(in, plan.parts, stream);
    else e = u16 ? norm_bwd_typed<float, uint16_t>(in, plan.parts, stream) : norm_bwd_typed<float, float>(in, plan.parts, stream);
    if (e != hipSuccess || a.dweight == nullptr) return e;
    norm_dweight_kernel<<<dim3(std::min((a.channels + 63) / 64, 1 << 16)), dim3(1024), 0, stream>>>(a.partials, plan.parts, a.channels, a.dweight);
    return hipGetLastError();
}

}  // namespace ssd
