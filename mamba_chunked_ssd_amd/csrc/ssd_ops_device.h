// ssd_ops_device.h -- device helpers of the short causal convolution and the
// selective scan: vectors of stored elements, the logistic function and
// softplus, and lane moves within the lanes that share a channel.
#pragma once

#include <type_traits>

#include "ssd_device.h"

namespace ssd {

constexpr uint32_t kNowhere = 0x7fffff00u;  // an offset behind any raw buffer here: such loads read 0, stores are dropped

// A raw buffer whose base is the same in every lane.  Said so outright: where
// the compiler cannot see it, it wraps every access in a loop over the lanes'
// values.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t uniform_rsrc(const void *base, uint32_t bytes) {
    const uint64_t a = reinterpret_cast<uint64_t>(base);
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
    return buffer_rsrc(reinterpret_cast<const void *>((uint64_t)hi << 32 | lo), __builtin_amdgcn_readfirstlane(bytes));
}

// V stored elements as one load, from memory or a raw buffer; unpack widens
// them exactly.
template <typename T, int V>
struct Raw;
template <>
struct Raw<float, 1> {
    float v;
    __device__ void zero() { v = 0.f; }
    __device__ void load(const float *p) { v = *p; }
    __device__ void load(__amdgpu_buffer_rsrc_t r, uint32_t off) { v = buffer_load_f32(r, (int)off); }
    __device__ void unpack(float (&f)[1]) const { f[0] = v; }
};
template <>
struct Raw<float, 4> {
    floatx4 v;
    __device__ void zero() { v = zero4(); }
    __device__ void load(const float *p) { v = *reinterpret_cast<const floatx4 *>(p); }
    __device__ void load(__amdgpu_buffer_rsrc_t r, uint32_t off) {
        v = __builtin_bit_cast(floatx4, buffer_load_x4(r, (int)off));
    }
    __device__ void unpack(float (&f)[4]) const {
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = v[e];
    }
};
template <>
struct Raw<uint16_t, 1> {
    uint32_t v;
    __device__ void zero() { v = 0; }
    __device__ void load(const uint16_t *p) { v = *p; }
    __device__ void load(__amdgpu_buffer_rsrc_t r, uint32_t off) {
        v = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, (int)off, 0, 0);
    }
    __device__ void unpack(float (&f)[1]) const { f[0] = bf16_to_f32(v); }
};
template <>
struct Raw<uint16_t, 4> {
    u32x2 v;
    __device__ void zero() { v = u32x2{0, 0}; }
    __device__ void load(const uint16_t *p) { v = *reinterpret_cast<const u32x2 *>(p); }
    __device__ void load(__amdgpu_buffer_rsrc_t r, uint32_t off) {
        v = __builtin_amdgcn_raw_buffer_load_b64(r, (int)off, 0, 0);
    }
    __device__ void unpack(float (&f)[4]) const {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            f[2 * e] = bf16lo(v[e]);
            f[2 * e + 1] = bf16hi(v[e]);
        }
    }
};
// V values stored as T (bf16: one rounding to nearest even, the output's own
// type; sums before it are fp32), to memory or to a raw buffer, which drops
// what falls outside.
template <int V>
__device__ __forceinline__ void store_n(float *p, const float (&f)[V]) {
    if constexpr (V == 1) *p = f[0];
    else *reinterpret_cast<floatx4 *>(p) = floatx4{f[0], f[1], f[2], f[3]};
}
template <int V>
__device__ __forceinline__ void store_n(uint16_t *p, const float (&f)[V]) {
    if constexpr (V == 1) *p = (uint16_t)(pack_bf16(f[0], 0.f) & 0xffffu);
    else *reinterpret_cast<u32x2 *>(p) = u32x2{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3])};
}
template <int V>
__device__ __forceinline__ void store_n(const float *, __amdgpu_buffer_rsrc_t r, uint32_t off, const float (&f)[V]) {
    if constexpr (V == 1)
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(f[0]), r, (int)off, 0, 0);
    else
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, floatx4{f[0], f[1], f[2], f[3]}), r, (int)off, 0,
                                               0);
}
template <int V>
__device__ __forceinline__ void store_n(const uint16_t *, __amdgpu_buffer_rsrc_t r, uint32_t off, const float (&f)[V]) {
    if constexpr (V == 1)
        __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(pack_bf16(f[0], 0.f) & 0xffffu), r, (int)off, 0, 0);
    else
        __builtin_amdgcn_raw_buffer_store_b64(u32x2{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3])}, r, (int)off, 0, 0);
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
// reciprocal is the limit 0.  The exponent is rounded to fp32, which puts the
// exponential off by |v| 2^-24 or so: an absolute error of 0.54 2^-24 at most in
// v logistic(v), of 0.27 2^-24 in logistic(v), though relative to the small
// values of negative v it grows with |v|.  Corrected as in softplus, the
// convolution's backward pass took 11 % more (4 x 4096 tokens of 5376 channels,
// bf16), the scan's 2 %.
__device__ __forceinline__ float logistic(float v) {
    return __builtin_amdgcn_rcpf(1.f + fast_exp2(-kLog2e * v));
}

// log(1 + exp(v)) = max(v, 0) + log1p(e), e = exp(-|v|) in (0, 1].  u = 1 + e
// drops low bits of e; e - (u - 1) is that loss exactly, and to first order
// log1p(e) = log(u) + (e - (u - 1)) / u, where / u matters only once the loss
// itself is below half a unit of log(u)'s last place.  So step sizes near
// 1e-3, which come from small e, keep their relative accuracy.
__device__ __forceinline__ float softplus(float v) {
    // exp(-|v|) = 2^t exp(-|v| - t log(2)): the exponent t rounded to fp32 would leave a relative error of |v| 2^-24,
    // to first order the second factor takes it back (held finite where v is infinite; a NaN stays one)
    const float t = -kLog2e * __builtin_fabsf(v);
    const float rest = __builtin_amdgcn_fmed3f(fmaf(t, -0.6931471805599453f, -__builtin_fabsf(v)), -1.f, 1.f);
    const float raw = fast_exp2(t), e = fmaf(raw, rest, raw);
    const float u = 1.f + e;
    const float lost = e - (u - 1.f);
    return fmaf(__builtin_amdgcn_logf(u), 0.6931471805599453f, lost) + fmaxf(v, 0.f);
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

// Sums over the channels of a wave, each channel on LPC neighbouring lanes:
// v[q][r], r < 4, is a lane's value number r of sum q.  Each step adds two
// lanes' values and hands one half of the sums to each, so a lane ends with
// one value a sum: that of r = channel_sum_r(lane), over the channels that lie
// on lanes of the same 64 / (16 .. 64) part.  Rows of 16 lanes hold 16 / LPC
// channels; within them a DPP add writes only the quads (bank_mask) that keep
// its half, two instructions for a pair of values.  (The matrix units would
// take the sum over lanes too, but fp32 products run on the vector units'
// time: 41 cycles each beside 4.4 for a fused multiply-add, measured, with
// nothing gained by interleaving.)
template <int LPC>
__device__ __forceinline__ int channel_sum_r(int lane) {
    if constexpr (LPC == 4) return lane >> 2 & 3;
    else if constexpr (LPC == 8) return (lane >> 4 & 1) + 2 * (lane >> 3 & 1);
    else return (lane >> 4 & 1) + 2 * (lane >> 5 & 1);
}
// Which part a lane's sum covers, of 64 / (4 LPC).
template <int LPC>
__device__ __forceinline__ int channel_sum_part(int lane) {
    return LPC == 4 ? lane >> 4 : LPC == 8 ? lane >> 5 : 0;
}
template <int LPC>
__device__ __forceinline__ void channel_sums(const float (&v)[2][4], float &s0, float &s1) {
    if constexpr (LPC == 4) {
        float a, b, c, d;
        // lanes 8-15 of a row keep r + 2, then odd quads r + 1.  A DPP operand must have been written two
        // instructions before: the nop covers the values coming in, the order those within.
        asm("s_nop 1\n\t"
            "v_add_f32_dpp %2, %6, %6 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
            "v_add_f32_dpp %2, %8, %8 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
            "v_add_f32_dpp %3, %7, %7 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
            "v_add_f32_dpp %3, %9, %9 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
            "v_add_f32_dpp %4, %10, %10 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
            "v_add_f32_dpp %4, %12, %12 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
            "v_add_f32_dpp %5, %11, %11 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
            "v_add_f32_dpp %5, %13, %13 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
            "v_add_f32_dpp %0, %2, %2 row_shl:4 row_mask:0xf bank_mask:0x5\n\t"
            "v_add_f32_dpp %0, %3, %3 row_shr:4 row_mask:0xf bank_mask:0xa\n\t"
            "v_add_f32_dpp %1, %4, %4 row_shl:4 row_mask:0xf bank_mask:0x5\n\t"
            "v_add_f32_dpp %1, %5, %5 row_shr:4 row_mask:0xf bank_mask:0xa"
            : "=&v"(s0), "=&v"(s1), "=&v"(a), "=&v"(b), "=&v"(c), "=&v"(d)
            : "v"(v[0][0]), "v"(v[0][1]), "v"(v[0][2]), "v"(v[0][3]), "v"(v[1][0]), "v"(v[1][1]), "v"(v[1][2]),
              "v"(v[1][3]));
    } else {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            float x, y;
            if constexpr (LPC == 8) {
                const bool upper = (threadIdx.x & 8) != 0;
                const float a = v[q][0] + lane_swap<8>(v[q][0]), b = v[q][2] + lane_swap<8>(v[q][2]);
                const float c = v[q][1] + lane_swap<8>(v[q][1]), d = v[q][3] + lane_swap<8>(v[q][3]);
                x = upper ? b : a;
                y = upper ? d : c;
            } else {
                // lanes 32-63 of the first and 0-31 of the second change places
                const auto e = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[q][0]), __float_as_uint(v[q][2]),
                                                                false, false);
                const auto o = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[q][1]), __float_as_uint(v[q][3]),
                                                                false, false);
                x = __uint_as_float(e[0]) + __uint_as_float(e[1]);
                y = __uint_as_float(o[0]) + __uint_as_float(o[1]);
            }
            // odd rows of the first and even rows of the second change places
            const auto w = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(y), false, false);
            (q == 0 ? s0 : s1) = __uint_as_float(w[0]) + __uint_as_float(w[1]);
        }
    }
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
