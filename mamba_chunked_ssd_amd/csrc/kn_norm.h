// kn_norm.h -- what the RMS norm's forward and backward kernels share: pieces
// of eight channels at any alignment, sums over the lanes of a row, where a row
// lies.
#pragma once

#include "ssd_launch.h"
#include "ssd_ops_device.h"
#include "ssd_ops_internal.h"

namespace ssd {
// Eight consecutive elements as they are stored, at any alignment of their type.
template <typename T>
struct Eight;
template <>
struct Eight<uint16_t> {
    u32x4 v;
    __device__ void zero() { v = u32x4{0, 0, 0, 0}; }
    __device__ void load(const uint16_t *p) { __builtin_memcpy(&v, p, 16); }
    __device__ void load_some(const uint16_t *p, int n) {
        zero();
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (e < n) v[e / 2] |= (uint32_t)p[e] << (16 * (e & 1));
    }
    __device__ float get(int e) const { return (e & 1) != 0 ? bf16hi(v[e / 2]) : bf16lo(v[e / 2]); }
};
template <>
struct Eight<float> {
    floatx4 v[2];
    __device__ void zero() { v[0] = v[1] = zero4(); }
    __device__ void load(const float *p) { __builtin_memcpy(v, p, 32); }
    __device__ void load_some(const float *p, int n) {
        zero();
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (e < n) v[e / 4][e % 4] = p[e];
    }
    __device__ float get(int e) const { return v[e / 4][e % 4]; }
};

// A row's piece at c0; LAST: it may end inside the piece or before it (what lies behind counts as 0).
template <bool LAST, typename T>
__device__ __forceinline__ void load_piece(Eight<T> &r, const T *row, int c0, int C) {
    if (!LAST || c0 + 8 <= C) r.load(row + c0);
    else if (c0 < C) r.load_some(row + c0, C - c0);
    else r.zero();
}

__device__ __forceinline__ void store_eight(uint16_t *p, const float (&f)[8]) {
    const u32x4 v = {pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])};
    __builtin_memcpy(p, &v, 16);
}
__device__ __forceinline__ void store_eight(float *p, const float (&f)[8]) { __builtin_memcpy(p, f, 32); }
// Codes of e4m3 (round to nearest even; every value is within 448 or a NaN).
__device__ __forceinline__ u32x2 codes_of(const float (&f)[8]) {
    u32x2 r;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * h], f[4 * h + 1], 0, false);
        r[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[4 * h + 2], f[4 * h + 3], lo, true);
    }
    return r;
}
__device__ __forceinline__ void store_eight(uint8_t *p, const float (&f)[8]) {
    const u32x2 v = codes_of(f);
    __builtin_memcpy(p, &v, 8);
}
__device__ __forceinline__ void store_at(uint16_t *p, float f) { *p = (uint16_t)(pack_bf16(f, 0.f) & 0xffffu); }
__device__ __forceinline__ void store_at(float *p, float f) { *p = f; }
__device__ __forceinline__ void store_at(uint8_t *p, float f) {
    *p = (uint8_t)(__builtin_amdgcn_cvt_pk_fp8_f32(f, 0.f, 0, false) & 0xff);
}
// The piece at c0 of a row (one rounding to nearest even where T has fewer bits).
template <bool LAST, typename T>
__device__ __forceinline__ void store_piece(T *row, int c0, int C, const float (&f)[8]) {
    if (!LAST || c0 + 8 <= C) {
        store_eight(row + c0, f);
    } else {
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (c0 + e < C) store_at(row + c0 + e, f[e]);
    }
}
template <bool LAST>
__device__ __forceinline__ void store_as(Stored t, void *base, int64_t at, int c0, int C, const float (&f)[8]) {
    if (t == Stored::bf16) store_piece<LAST>(static_cast<uint16_t *>(base) + at, c0, C, f);
    else if (t == Stored::f32) store_piece<LAST>(static_cast<float *>(base) + at, c0, C, f);
    else store_piece<LAST>(static_cast<uint8_t *>(base) + at, c0, C, f);
}
// A row behind its sequence's end.
template <int TPR>
__device__ __forceinline__ void zero_row(Stored t, void *base, int64_t at, int C) {
    const float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int c0 = threadIdx.x % TPR * 8; c0 < C; c0 += TPR * 8) store_as<true>(t, base, at, c0, C, z);
}

// Larger of two magnitudes given by their bits, a NaN above all.
__device__ __forceinline__ float larger(float a, float b) {
    return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b)));
}
__device__ __forceinline__ double larger(double a, double b) {
    return __longlong_as_double(max(__double_as_longlong(a), __double_as_longlong(b)));
}

// The sum, or the largest magnitude, over the threads that hold a row: a wave,
// or a block of four with `room` in LDS.  Reductions follow one another, so the
// rooms alternate: a wave writes one again only after the next one's barrier.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float *room) {
    v = lane_total<16>(v);
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
    const auto t = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(t[0]) + __uint_as_float(t[1]);
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) room[threadIdx.x >> 6] = v;
        __syncthreads();
        v = (room[0] + room[1]) + (room[2] + room[3]);
    }
    return v;
}
template <int TPR>
__device__ __forceinline__ float row_most(float v, float *room) {
    v = larger(v, lane_swap<1>(v));
    v = larger(v, lane_swap<2>(v));
    v = larger(v, lane_swap<4>(v));
    v = larger(v, lane_swap<8>(v));
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = larger(__uint_as_float(s[0]), __uint_as_float(s[1]));
    const auto t = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = larger(__uint_as_float(t[0]), __uint_as_float(t[1]));
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) room[threadIdx.x >> 6] = v;
        __syncthreads();
        v = larger(larger(room[0], room[1]), larger(room[2], room[3]));
    }
    return v;
}

// f(i, whether the piece is a row's last) for its NV pieces.
template <int NV, typename F>
__device__ __forceinline__ void for_pieces(F &&f) {
    for_lanes<NV>([&](auto i) { f(i, std::integral_constant<bool, decltype(i)::value + 1 == NV>{}); });
}

// f(integral constant n), n in LO .. HI (host).
template <int LO, int HI, typename F>
inline void with_pieces(int n, F &&f) {
    if constexpr (LO < HI) {
        if (n > LO) return with_pieces<LO + 1, HI>(n, static_cast<F &&>(f));
    }
    f(std::integral_constant<int, LO>{});
}

// Where a row lies; rows are taken in turn by waves or blocks.
struct Place {
    int64_t b, t;
    bool live;
};
__device__ __forceinline__ Place place_of(uint32_t row, uint32_t L, const int32_t *lengths) {
    const uint32_t b = row / L, t = row - b * L;
    return Place{b, t, lengths == nullptr || (int64_t)t < (int64_t)max(lengths[b], 0)};
}

}  // namespace ssd
