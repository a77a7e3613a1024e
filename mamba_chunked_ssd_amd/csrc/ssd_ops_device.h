// ssd_ops_device.h -- device helpers of the short causal convolution and the
// selective scan: vectors of stored elements, the logistic function and
// softplus, and lane moves within the lanes that share a channel.
#pragma once

#include <type_traits>

#include "ssd_device.h"

namespace ssd {

// V stored elements as one load; unpack widens them exactly.
template <typename T, int V>
struct Raw;
template <>
struct Raw<float, 1> {
    float v;
    __device__ void zero() { v = 0.f; }
    __device__ void load(const float *p) { v = *p; }
    __device__ void unpack(float (&f)[1]) const { f[0] = v; }
};
template <>
struct Raw<float, 4> {
    floatx4 v;
    __device__ void zero() { v = zero4(); }
    __device__ void load(const float *p) { v = *reinterpret_cast<const floatx4 *>(p); }
    __device__ void unpack(float (&f)[4]) const {
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = v[e];
    }
};
template <>
struct Raw<float, 8> {
    floatx4 v[2];
    __device__ void zero() { v[0] = v[1] = zero4(); }
    __device__ void load(const float *p) {
        v[0] = *reinterpret_cast<const floatx4 *>(p);
        v[1] = *reinterpret_cast<const floatx4 *>(p + 4);
    }
    __device__ void unpack(float (&f)[8]) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = v[e / 4][e % 4];
    }
};
template <>
struct Raw<uint16_t, 1> {
    uint32_t v;
    __device__ void zero() { v = 0; }
    __device__ void load(const uint16_t *p) { v = *p; }
    __device__ void unpack(float (&f)[1]) const { f[0] = bf16_to_f32(v); }
};
template <>
struct Raw<uint16_t, 4> {
    u32x2 v;
    __device__ void zero() { v = u32x2{0, 0}; }
    __device__ void load(const uint16_t *p) { v = *reinterpret_cast<const u32x2 *>(p); }
    __device__ void unpack(float (&f)[4]) const {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            f[2 * e] = bf16lo(v[e]);
            f[2 * e + 1] = bf16hi(v[e]);
        }
    }
};
template <>
struct Raw<uint16_t, 8> {
    u32x4 v;
    __device__ void zero() { v = u32x4{0, 0, 0, 0}; }
    __device__ void load(const uint16_t *p) { v = *reinterpret_cast<const u32x4 *>(p); }
    __device__ void unpack(float (&f)[8]) const {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f[2 * e] = bf16lo(v[e]);
            f[2 * e + 1] = bf16hi(v[e]);
        }
    }
};

// V values stored as T (bf16: one rounding to nearest even, the output's own
// type; sums before it are fp32).
template <int V>
__device__ __forceinline__ void store_n(float *p, const float (&f)[V]) {
    if constexpr (V == 1) {
        *p = f[0];
    } else {
#pragma unroll
        for (int e = 0; e < V; e += 4)
            *reinterpret_cast<floatx4 *>(p + e) = floatx4{f[e], f[e + 1], f[e + 2], f[e + 3]};
    }
}
template <int V>
__device__ __forceinline__ void store_n(uint16_t *p, const float (&f)[V]) {
    if constexpr (V == 1) {
        *p = (uint16_t)(pack_bf16(f[0], 0.f) & 0xffffu);
    } else if constexpr (V == 4) {
        *reinterpret_cast<u32x2 *>(p) = u32x2{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3])};
    } else {
        *reinterpret_cast<u32x4 *>(p) = u32x4{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                                              pack_bf16(f[6], f[7])};
    }
}

template <typename T>
__device__ __forceinline__ float load_one(const T *p, int64_t i) {
    float f[1];
    Raw<T, 1> r;
    r.load(p + i);
    r.unpack(f);
    return f[0];
}

// 1 / (1 + exp(-v)); exp2 overflows to infinity for very negative v, whose
// reciprocal is the limit 0.
__device__ __forceinline__ float logistic(float v) {
    return __builtin_amdgcn_rcpf(1.f + fast_exp2(-kLog2e * v));
}

// log(1 + exp(v)) = max(v, 0) + log1p(e), e = exp(-|v|) in (0, 1], and
// log1p(e) = 2 atanh(s), s = e / (2 + e) <= 1/3, by the odd series of atanh to
// s^15 (the rest is below 1e-9 of the sum).  1 + e is never formed, so small e
// keep their relative accuracy: step sizes near 1e-3 come from such e.
__device__ __forceinline__ float softplus(float v) {
    const float e = fast_exp2(-kLog2e * __builtin_fabsf(v));
    const float s = e * __builtin_amdgcn_rcpf(2.f + e);
    const float q = s * s;
    float r = 1.f / 15.f;
    r = fmaf(r, q, 1.f / 13.f);
    r = fmaf(r, q, 1.f / 11.f);
    r = fmaf(r, q, 1.f / 9.f);
    r = fmaf(r, q, 1.f / 7.f);
    r = fmaf(r, q, 1.f / 5.f);
    r = fmaf(r, q, 1.f / 3.f);
    r = fmaf(r, q, 1.f);
    return fmaf(2.f * s, r, fmaxf(v, 0.f));
}

// v moved by one DPP control (every lane of the controls used has a source).
template <int CTRL>
__device__ __forceinline__ float dpp_f32(float v) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, 0xf, 0xf, true));
}
// As above in the banks (quads of each row of 16 lanes) of the mask, old elsewhere.
template <int CTRL, int BANKS>
__device__ __forceinline__ float dpp_banks_f32(float old, float v) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp((int)__float_as_uint(old), (int)__float_as_uint(v), CTRL,
                                                                 0xf, BANKS, false));
}

// Lane K's value of each group of LPC consecutive lanes.
template <int LPC, int K>
__device__ __forceinline__ float lane_bcast(float v) {
    if constexpr (LPC == 2) {
        return dpp_f32<K | (K << 2) | ((K + 2) << 4) | ((K + 2) << 6)>(v);  // quad_perm
    } else if constexpr (LPC == 4) {
        return dpp_f32<K * 0x55>(v);  // quad_perm
    } else if constexpr (LPC == 8) {
        // row_newbcast: one lane of each row of 16 to the whole row, then to its upper half
        return dpp_banks_f32<0x158 + K, 0xc>(dpp_f32<0x150 + K>(v), v);
    } else {
        return dpp_f32<0x150 + K>(v);  // row_newbcast
    }
}

// The value of the lane whose index differs in bit BIT of a group of LPC (for
// BIT 4, in all three low bits: a lane of the same pair once the sums over
// bits 1 and 2 are taken).
template <int BIT>
__device__ __forceinline__ float lane_swap(float v) {
    if constexpr (BIT == 1) return dpp_f32<0xB1>(v);        // quad_perm 1,0,3,2
    else if constexpr (BIT == 2) return dpp_f32<0x4E>(v);   // quad_perm 2,3,0,1
    else if constexpr (BIT == 4) return dpp_f32<0x141>(v);  // row_half_mirror
    else return dpp_f32<0x128>(v);                          // row_ror:8
}

// p[k], k < LPC, summed over the LPC lanes of a group; lane j returns the sum
// of p[j].  Halves the values at each step, so LPC - 1 steps for LPC sums.
template <int LPC>
__device__ __forceinline__ float lane_sums(float (&p)[LPC], int j) {
    if constexpr (LPC == 1) {
        return p[0];
    } else {
        constexpr int H = LPC / 2;
        float q[H];
        const bool upper = (j & H) != 0;
#pragma unroll
        for (int k = 0; k < H; ++k) {
            const float lo = p[k] + lane_swap<H>(p[k]);
            const float hi = p[k + H] + lane_swap<H>(p[k + H]);
            q[k] = upper ? hi : lo;
        }
        return lane_sums<H>(q, j);
    }
}

// One value summed over the LPC lanes of a group, in every lane.
template <int LPC>
__device__ __forceinline__ float lane_total(float v) {
    if constexpr (LPC >= 16) v += lane_swap<8>(v);
    if constexpr (LPC >= 8) v += lane_swap<4>(v);
    if constexpr (LPC >= 4) v += lane_swap<2>(v);
    v += lane_swap<1>(v);
    return v;
}

// f(integral constant k) for k = 0 .. N - 1 (DPP controls are immediates).
template <int N, typename F, int K = 0>
__device__ __forceinline__ void for_lanes(F &&f) {
    if constexpr (K < N) {
        f(std::integral_constant<int, K>{});
        for_lanes<N, F, K + 1>(static_cast<F &&>(f));
    }
}

}  // namespace ssd
