// kn_norm.hip -- the root-mean-square norm before a layer's projection, with
// the residual's addition, also into 8 bits with scales.
//
//   u = x + residual ,  r = (mean u^2 + eps)^-1/2 ,  y = u r w
//
// Bound by memory: every element comes once and goes once against some ten
// vector operations, so a row stays in registers between its sum and its
// output.  Up to 4096 channels a wave holds a row, eight channels a lane and
// piece, and sums by lane moves alone; up to 16384 a block of four waves does,
// through LDS once a row (twice with a scale for the row); longer rows are read twice (the second time from the
// caches).  Rows need no alignment: the loads of 16 bytes are unaligned ones
// where they must be, and only a row's last channels (channels mod 8) come one
// by one.
//
// Measured: 8 x 4096 tokens of 2560 channels, bf16 with an fp32 stream, into e4m3
// with a scale to 128 columns 165 us, 5.6 TB/s (a large copy: 5.1); 3 x 517
// tokens of 771 fp32 channels 5.5 us; one token of 2560 4.8 us, a call 13.
#include <algorithm>

#include "kn_norm.h"

namespace ssd {
namespace {

constexpr float kE4m3Max = 448.f, kLeastScale = 1.1754943508222875e-38f;

struct NormIn {
    const void *x, *residual;
    const float *weight;
    const int32_t *lengths;
    void *y, *residual_out;
    float *scales;
    Strides xs, rs;
    uint32_t rows;
    int L, C, nscale, block;
    float eps;
    Stored res, out;
};

// y of one piece into f, or with codes y / scale: the lanes of a block of
// columns are neighbours, 4, 8 or 16 of them.
__device__ __forceinline__ void quantise(const NormIn &a, float (&f)[8], int64_t row, int c0, float row_scale) {
    float scale = row_scale;
    if (a.block != 0) {
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = larger(m, __builtin_fabsf(f[e]));
        m = larger(m, lane_swap<1>(m));
        m = larger(m, lane_swap<2>(m));
        if (a.block >= 64) m = larger(m, lane_swap<4>(m));
        if (a.block >= 128) m = larger(m, lane_swap<8>(m));
        scale = larger(m / kE4m3Max, kLeastScale);
        if (c0 < a.C && c0 % a.block == 0) a.scales[row * a.nscale + c0 / a.block] = scale;
    }
    const float inv = 1.f / scale;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float q = f[e] * inv;
        // the scale's own rounding may leave the largest just above 448; a NaN stays one
        f[e] = q > kE4m3Max ? kE4m3Max : q < -kE4m3Max ? -kE4m3Max : q;
    }
}

template <typename TX, typename TR, int TPR, int NV>
__global__ __launch_bounds__(256) void norm_fwd_kernel(const NormIn a) {
    constexpr bool kRes = !std::is_same<TR, void>::value;
    typedef typename std::conditional<kRes, TR, float>::type R;
    __shared__ float room[2][4];
    const int lane = threadIdx.x % TPR, C = a.C;
    uint32_t row = blockIdx.x, step = gridDim.x;
    if constexpr (TPR == 64) {
        row = row * 4 + (uint32_t)__builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
        step *= 4;
    }
    const auto at_piece = [&](int i) { return (i * TPR + lane) * 8; };
    int turn = 0;
    for (uint64_t at = row; at < a.rows; at += step) {
        const Place p = place_of((uint32_t)at, (uint32_t)a.L, a.lengths);
        const int64_t out = (int64_t)at * C;
        if (!p.live) {
            zero_row<TPR>(a.out, a.y, out, C);
            if (a.residual_out != nullptr) zero_row<TPR>(a.res, a.residual_out, out, C);
            if (a.out == Stored::e4m3)
                for (int k = lane; k < a.nscale; k += TPR) a.scales[(int64_t)at * a.nscale + k] = kLeastScale;
            continue;
        }
        Eight<TX> x[NV];
        Eight<R> res[NV];
        Eight<float> wt[NV];
        const TX *xr = static_cast<const TX *>(a.x) + p.b * a.xs.batch + p.t * a.xs.row;
        const R *rr = static_cast<const R *>(a.residual) + p.b * a.rs.batch + p.t * a.rs.row;
        for_pieces<NV>([&](auto i, auto last) { load_piece<last>(x[i], xr, at_piece(i), C); });
        if constexpr (kRes) for_pieces<NV>([&](auto i, auto last) { load_piece<last>(res[i], rr, at_piece(i), C); });
        if (a.weight != nullptr)
            for_pieces<NV>([&](auto i, auto last) { load_piece<last>(wt[i], a.weight, at_piece(i), C); });
        else
            for_pieces<NV>([&](auto i, auto) { wt[i].v[0] = wt[i].v[1] = floatx4{1.f, 1.f, 1.f, 1.f}; });
        float u[NV][8], sum = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                u[i][e] = x[i].get(e);
                if constexpr (kRes) u[i][e] += res[i].get(e);
                sum = fmaf(u[i][e], u[i][e], sum);
            }
        sum = row_sum<TPR>(sum, room[turn]);
        turn ^= 1;
        const float r = rsqrtf(sum / (float)C + a.eps);
        float row_scale = 0.f;
        if (a.out == Stored::e4m3 && a.block == 0) {
            // over y itself: u w alone, taken beside the sum, may leave fp32's range where y does not
            float most = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) most = larger(most, __builtin_fabsf(u[i][e] * r * wt[i].get(e)));
            row_scale = larger(row_most<TPR>(most, room[turn]) / kE4m3Max, kLeastScale);
            turn ^= 1;
            if (lane == 0) a.scales[at] = row_scale;
        }
        if (a.residual_out != nullptr)
            for_pieces<NV>([&](auto i, auto last) { store_as<last>(a.res, a.residual_out, out, at_piece(i), C, u[i]); });
        for_pieces<NV>([&](auto i, auto last) {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = u[i][e] * r * wt[i].get(e);
            if (a.out == Stored::e4m3) quantise(a, f, (int64_t)at, at_piece(i), row_scale);
            store_as<last>(a.out, a.y, out, at_piece(i), C, f);
        });
    }
}

// Rows of any length, a block each: once for the sum, once for the output.  A
// lane's sum is over up to 2^16 elements and is held in 64 bits, and so is, for
// the row's scale, the largest |u w|, whose product may leave fp32's range where
// y does not.
template <typename TX, typename TR>
__global__ __launch_bounds__(256) void norm_fwd_long_kernel(const NormIn a) {
    constexpr bool kRes = !std::is_same<TR, void>::value;
    typedef typename std::conditional<kRes, TR, float>::type R;
    __shared__ float room[2][4];
    const int C = a.C;
    int turn = 0;
    for (uint64_t at = blockIdx.x; at < a.rows; at += gridDim.x) {
        const Place p = place_of((uint32_t)at, (uint32_t)a.L, a.lengths);
        const TX *xr = static_cast<const TX *>(a.x) + p.b * a.xs.batch + p.t * a.xs.row;
        const R *rr = static_cast<const R *>(a.residual) + p.b * a.rs.batch + p.t * a.rs.row;
        const int stop = p.live ? C : 0;
        const auto piece = [&](int c0, float (&u)[8], float (&w)[8]) {
            Eight<TX> x;
            Eight<R> res;
            Eight<float> v;
            load_piece<true>(x, xr, c0, stop);
            if constexpr (kRes) load_piece<true>(res, rr, c0, stop);
            if (a.weight != nullptr) load_piece<true>(v, a.weight, c0, stop);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                u[e] = x.get(e);
                if constexpr (kRes) u[e] += res.get(e);
                w[e] = a.weight != nullptr ? v.get(e) : 1.f;
            }
        };
        const bool by_row = a.out == Stored::e4m3 && a.block == 0;
        double total = 0.0, most = 0.0;
        float u[8], w[8];
        for (int c0 = threadIdx.x * 8; c0 < stop; c0 += 2048) {
            piece(c0, u, w);
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) s = fmaf(u[e], u[e], s);
            total += s;
            if (by_row) {
#pragma unroll
                for (int e = 0; e < 8; ++e) most = larger(most, __builtin_fabs((double)u[e] * (double)w[e]));
            }
        }
        const float sum = row_sum<256>((float)total, room[turn]);
        turn ^= 1;
        const float r = p.live ? rsqrtf(sum / (float)C + a.eps) : 0.f;
        float row_scale = 0.f;
        if (by_row) {
            row_scale = larger(row_most<256>(__builtin_fabsf((float)(most * (double)r)), room[turn]) / kE4m3Max, kLeastScale);
            turn ^= 1;
            if (threadIdx.x == 0) a.scales[at] = row_scale;
        }
        const int64_t out = (int64_t)at * C;
        // every lane takes every turn: a block of columns is shared by lanes
        for (int base = 0; base < C; base += 2048) {
            const int c0 = base + threadIdx.x * 8;
            piece(c0, u, w);
            if (a.residual_out != nullptr) store_as<true>(a.res, a.residual_out, out, c0, C, u);
#pragma unroll
            for (int e = 0; e < 8; ++e) u[e] = u[e] * r * w[e];
            if (a.out == Stored::e4m3) quantise(a, u, (int64_t)at, c0, row_scale);
            store_as<true>(a.out, a.y, out, c0, C, u);
        }
    }
}

template <typename TX, typename TR>
hipError_t norm_fwd_typed(const NormIn &a, hipStream_t stream) {
    const uint32_t most = 1u << 20;
    const dim3 block(256);
    if (a.C > kNormBlockRow) {
        norm_fwd_long_kernel<TX, TR><<<dim3(std::min(a.rows, most)), block, 0, stream>>>(a);
    } else if (a.C > kNormWaveRow) {
        const int nv = (a.C + 2047) / 2048;
        with_pieces<3, 8>(nv, [&](auto n) { norm_fwd_kernel<TX, TR, 256, n><<<dim3(std::min(a.rows, most)), block, 0, stream>>>(a); });
    } else {
        const int nv = (a.C + 511) / 512;
        with_pieces<1, 8>(nv, [&](auto n) { norm_fwd_kernel<TX, TR, 64, n><<<dim3(std::min((a.rows + 3) / 4, most)), block, 0, stream>>>(a); });
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_fwd(const NormArgs &a, hipStream_t stream) {
    const int nscale = a.scale_block == 0 ? 1 : (a.channels + a.scale_block - 1) / a.scale_block;
    const NormIn in{a.in,   a.residual, a.weight, a.lengths,  a.out,         a.residual_out, a.scales, a.xs, a.rs,
                    (uint32_t)(a.batch * a.seqlen), a.seqlen, a.channels, nscale, a.scale_block, a.eps, a.res, a.y};
    const bool x16 = a.x == Stored::bf16, r16 = a.res == Stored::bf16;
    if (a.residual == nullptr) return x16 ? norm_fwd_typed<uint16_t, void>(in, stream) : norm_fwd_typed<float, void>(in, stream);
    if (x16) return r16 ? norm_fwd_typed<uint16_t, uint16_t>(in, stream) : norm_fwd_typed<uint16_t, float>(in, stream);
    return r16 ? norm_fwd_typed<float, uint16_t>(in, stream) : norm_fwd_typed<float, float>(in, stream);
}

}  // namespace ssd
